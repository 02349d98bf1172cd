"""GPU parity of the serving operators (norm and rotation, packed causal
attention, the 8-bit paged cache, attention over it) against the fp64 oracle,
through the binding.

Tolerances, with u the unit roundoff of the 16-bit type (2^-11 fp16, 2^-8
bf16), S = sum of weight * |value| of a result and r the reference:
- norm and rotation: u |r| for the one rounding; the sine and cosine are
  within 2^-20 absolute, the fp32 arithmetic within 2^-20 relative, both of
  the pair's size sqrt(a^2 + b^2): 2^-18 of it in all.
- packed attention: each weight is rounded once (u S), the result once
  (u |r|), both half of that on the 2^-e significand grid at best and a whole
  u at worst, with 1/16 more for the products of errors; logits of size up to
  L (sum |q||k| scale) computed in fp32 over d terms are off by (d + 4) 2^-24 L
  and a weight by as much relative, twice that with the sum: 2 (d + 4) 2^-24 L S;
  the exponential is within 2^-21, and an fp16 weight below 2^-14 is off by up
  to 2^-25 of the row's largest: n 2^-25 max|v|.
- cache: equal codes and equal values.
- cache attention: as packed attention with u = 2^-11 for the weights
  whatever the type, the query's rounding to fp16 at 2^-25 of its largest
  value adding 2^-24 to the logits' relative error."""
import numpy as np
import pytest
import torch

import oracle
from helpers import lib

pytestmark = pytest.mark.gpu

F16, BF16 = oracle.F16, oracle.BF16
TD = {F16: torch.float16, BF16: torch.bfloat16}
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module")
def m():
    return lib()


def _rand(seed, *shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TD[dtype])


def _val(t):
    return t.cpu().to(torch.float64).numpy()


def _slices(rows, heads, d, dtype, pad):
    """A [rows][heads][d] device tensor with `pad` more values between rows, filled with NaN around it."""
    big = torch.full((rows, heads * d + pad), float("nan"), dtype=TD[dtype], device="cuda")
    return big[:, : heads * d].view(rows, heads, d) if pad == 0 else big[:, : heads * d].unflatten(1, (heads, d))


# ------------------------------------------------------------ norm and rotation

def _check_rope(got, x, pos, f, half, w, eps, mag, dtype, what):
    want = oracle.qk_norm_rope(_val(x), pos, f, half, w, eps, mag)
    n = len(f)
    size = np.abs(want)
    a, b = (slice(0, n), slice(n, 2 * n)) if half else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    pair = np.hypot(want[..., a], want[..., b])
    size[..., a], size[..., b] = pair, pair
    tol = U[dtype] * np.abs(want) + 2.0 ** -18 * size + (2.0 ** -25 if dtype == F16 else 0.0)
    bad = np.abs(_val(got) - want) / np.maximum(tol, 1e-300)
    assert np.all(bad <= 1), f"{what}: {bad.max():.3g} of the tolerance at {np.unravel_index(bad.argmax(), bad.shape)}"


@pytest.mark.parametrize("tokens,hq,hk,d,rot,half,norm,dtype", [
    (1, 4, 1, 128, 128, True, "qk", BF16), (17, 32, 8, 128, 128, True, "qk", F16), (700, 32, 8, 128, 128, True, "qk", BF16),
    (33, 3, 3, 64, 32, False, "", F16), (65, 5, 2, 96, 96, True, "q", F16), (65, 5, 2, 96, 40, False, "k", BF16),
    (9, 2, 1, 256, 256, True, "qk", BF16), (40, 7, 1, 256, 8, False, "qk", F16), (5, 1, 1, 8, 8, True, "qk", F16),
    (21, 2, 2, 16, 0, True, "qk", BF16), (1100, 12, 4, 64, 64, False, "qk", F16), (2000, 9, 7, 24, 24, True, "k", F16),
    (3000, 1, 1, 128, 64, True, "", BF16)])
def test_rope_matches_oracle(m, tokens, hq, hk, d, rot, half, norm, dtype):
    q, k = _rand(1, tokens, hq, d, dtype=dtype, scale=2.0), _rand(2, tokens, hk, d, dtype=dtype, scale=0.3)
    wq, wk = _rand(3, d, dtype=dtype) + 1, _rand(4, d, dtype=dtype)
    pos = torch.from_numpy(np.random.default_rng(5).integers(0, 200000, tokens).astype(np.int32))
    op = m.QKNormRope(hq, hk, d, rot_dim=rot, layout=m.ATTN_ROPE_HALF if half else m.ATTN_ROPE_INTERLEAVED,
                      dtype=m.GEMM_BF16 if dtype == BF16 else m.GEMM_F16, eps=1e-5, magnitude=1.25)
    qo, ko = _slices(tokens, hq, d, dtype, 8), _slices(tokens, hk, d, dtype, 0)
    op.run(q.cuda(), k.cuda(), pos.cuda(), qo, ko, wq.cuda() if "q" in norm else None, wk.cuda() if "k" in norm else None)
    torch.cuda.synchronize()
    f = oracle.rope_frequencies(rot, 10000.0) if rot else np.zeros(0)
    for got, x, w, on in ((qo, q, wq, "q" in norm), (ko, k, wk, "k" in norm)):
        _check_rope(got, x, pos.numpy(), f, half, _val(w) if on else None, 1e-5, 1.25, dtype, (tokens, hq, hk, d))


def test_rope_in_place_on_a_projection_and_extreme_positions(m):
    """Queries and keys are slices of one tensor, turned in place; its values stay; positions at both ends of int32."""
    t, hq, hk, d = 12, 4, 2, 128
    qkv = _rand(6, t, (hq + 2 * hk) * d, dtype=BF16).cuda()
    before = qkv.clone()
    q, k = qkv[:, : hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131071, 1 << 20, 7, 8, 9, 10, 11], dtype=np.int32)
    op = m.QKNormRope(hq, hk, d, dtype=m.GEMM_BF16, base=500000.0, factor=8.0, context=8192.0, low_turns=1.0, high_turns=4.0)
    f = np.array(m.attn_rope_frequencies(op.desc))
    op.run(q, k, torch.from_numpy(pos).cuda(), q, k)
    torch.cuda.synchronize()
    x = before[:, : hq * d].unflatten(1, (hq, d)).cpu()
    # (fp64 itself holds an angle of 2^31 radians to 2^-22, and the frequencies' 2^-53 grows to as much)
    _check_rope(q, x, pos, f, True, None, 0.0, 1.0, BF16, "in place")
    assert torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_rope_own_frequencies_and_no_tokens(m):
    f = [0.5, 0.25, -0.1, 7.5]
    op = m.QKNormRope(2, 1, 64, rot_dim=8, layout=m.ATTN_ROPE_INTERLEAVED, dtype=m.GEMM_F16, frequencies=f)
    q, k, pos = _rand(7, 10, 2, 64, dtype=F16), _rand(8, 10, 1, 64, dtype=F16), np.arange(10, dtype=np.int32) * 100
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    op.run(q.cuda(), k.cuda(), torch.from_numpy(pos).cuda(), qo, ko)
    _check_rope(qo, q, pos, np.array(f), False, None, 0.0, 1.0, F16, "own")
    assert torch.equal(ko[:, :, 8:].cpu(), k[:, :, 8:])
    op.run(qo[:0], ko[:0], torch.empty(0, dtype=torch.int32, device="cuda"), qo[:0], ko[:0])


def test_rope_zero_rows_and_nan_stay_in_their_heads(m):
    q = torch.zeros(3, 2, 64, dtype=torch.float16)
    q[1, 0, 5], q[2, 1, 3] = float("nan"), float("inf")
    k = torch.ones(3, 1, 64, dtype=torch.float16)
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    op = m.QKNormRope(2, 1, 64, dtype=m.GEMM_F16)
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    op.run(q.cuda(), k.cuda(), torch.arange(3, dtype=torch.int32).cuda(), qo, ko, w, w)
    qo = qo.cpu()
    assert not qo[0].any() and not qo[1, 1].any() and not qo[2, 0].any()
    assert qo[1, 0].isnan().all() and torch.isfinite(ko).all()


# ------------------------------------------------------------ packed attention

def _cu(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def _attention_tol(dtype_out, u_w, want, mag, logit, n, vmax, extra=0.0):
    u = U[dtype_out]
    return (1 + 2.0 ** -4) * (u * np.abs(want) + (u_w + 2.0 ** -21) * mag) + 2 * (logit + extra) * mag + n * 2.0 ** -25 * vmax


def _run_prompt(m, q, k, v, cu_q, cu_k, dtype, causal=True, scale=0.0, pad=0):
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    op = m.PromptAttention(hq, hk, d, dtype=m.GEMM_BF16 if dtype == BF16 else m.GEMM_F16, causal=causal, scale=scale)
    dev = []
    for x in (q, k, v):
        s = _slices(x.shape[0], x.shape[1], d, dtype, pad)
        s.copy_(x)
        dev.append(s)
    out = _slices(q.shape[0], hq, d, dtype, pad)
    op.run(*dev, torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda(), out)
    assert op.sync_status() == m.GEMM_OK
    op.close()
    return out


def _check_prompt(got, q, k, v, cu_q, cu_k, dtype, causal=True, scale=None, what=""):
    d = q.shape[2]
    want, mag = oracle.prompt_attention(_val(q), _val(k), _val(v), cu_q, cu_k, causal, scale)
    s = 1 / np.sqrt(d) if scale is None else scale
    big = np.sqrt((_val(q) ** 2).sum(-1).max() * max((_val(k) ** 2).sum(-1).max() if k.numel() else 0, 1e-9)) * s
    vmax = float(v.abs().max()) if v.numel() else 0.0
    tol = _attention_tol(dtype, U[dtype], want, mag, (d + 4) * 2.0 ** -24 * big, max(k.shape[0], 1), vmax)
    used = np.zeros(q.shape[0], dtype=bool)
    for a, b in zip(cu_q[:-1], cu_q[1:]):
        used[a:b] = True
    diff = np.abs(_val(got) - want)[used]
    assert np.all(np.isfinite(diff)), what
    bad = diff / np.maximum(tol[used], 1e-30)
    assert np.all(bad <= 1), f"{what}: {bad.max():.3g} of the tolerance"


@pytest.mark.parametrize("lens,hq,hk,d,dtype", [
    ([1], 1, 1, 128, BF16), ([128], 1, 1, 64, F16), ([129, 1, 127, 300], 2, 2, 128, F16), ([5, 260, 64], 8, 2, 128, BF16),
    ([33, 77], 12, 4, 64, F16), ([50, 3], 7, 1, 64, BF16), ([40], 48, 1, 128, F16), ([9, 2], 128, 1, 64, BF16),
    ([600], 4, 4, 128, BF16), ([513], 3, 3, 64, F16), ([1] * 70 + [200], 4, 2, 64, F16)])
def test_prompt_matches_oracle(m, lens, hq, hk, d, dtype):
    cu, n = _cu(lens), sum(lens)
    q, k, v = (_rand(10 + i, n, h, d, dtype=dtype) for i, h in enumerate((hq, hk, hk)))
    _check_prompt(_run_prompt(m, q, k, v, cu, cu, dtype), q, k, v, cu, cu, dtype, what=str((lens, hq, hk, d)))


@pytest.mark.parametrize("nq,nk,causal,pad", [
    ([3, 1, 130], [400, 129, 257], True, 0),          # a later piece of a prompt; single queries
    ([200, 64, 0, 5], [70, 0, 9, 3], True, 8),        # queries before every key, no keys, no queries
    ([200, 64, 0, 5], [70, 0, 9, 130], False, 64),    # all keys
    ([1, 1, 1, 1, 1], [1, 127, 128, 129, 500], True, 0)])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16)])
def test_prompt_lengths_of_keys(m, nq, nk, causal, pad, d, dtype):
    cu_q, cu_k = _cu(nq), _cu(nk)
    q, k, v = _rand(20, sum(nq), 6, d, dtype=dtype), _rand(21, sum(nk), 2, d, dtype=dtype), _rand(22, sum(nk), 2, d, dtype=dtype)
    got = _run_prompt(m, q, k, v, cu_q, cu_k, dtype, causal=causal, scale=0.2, pad=pad)
    _check_prompt(got, q, k, v, cu_q, cu_k, dtype, causal, float(np.float32(0.2)), str((nq, nk)))


def test_prompt_rows_of_no_sequence_are_left(m):
    q, k, v = (_rand(30 + i, 40, 2, 64, dtype=F16) for i in range(3))
    cu = np.array([0, 10, 25], dtype=np.int32)
    got = _run_prompt(m, q, k, v, cu, cu, F16)
    assert got[25:].isnan().all()
    _check_prompt(got, q, k, v, cu, cu, F16)
    # lengths past the tensors are cut
    wild = np.array([0, 10, 4000], dtype=np.int32)
    cut = np.array([0, 10, 40], dtype=np.int32)
    _check_prompt(_run_prompt(m, q, k, v, wild, wild, F16), q, k, v, cut, cut, F16)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_nothing_leaks_between_sequences(m, d):
    """The middle sequence is infinities and NaN: its neighbours' results are those without it."""
    lens = [70, 45, 131]
    cu, n = _cu(lens), sum(lens)
    q, k, v = (_rand(40 + i, n, 4 if i == 0 else 2, d, dtype=BF16) for i in range(3))
    clean = _run_prompt(m, q, k, v, cu, cu, BF16)
    for x in (q, k, v):
        x[70:115] = torch.tensor([float("inf"), float("nan"), float("-inf")]).repeat(15)[:, None, None]
    dirty = _run_prompt(m, q, k, v, cu, cu, BF16)
    for rows in (slice(0, 70), slice(115, n)):
        assert torch.equal(clean[rows], dirty[rows])


def test_prompt_masked_keys_may_hold_anything(m):
    """A later key's NaN does not reach an earlier query of its sequence, nor does a later value's."""
    cu = _cu([200])
    q, k, v = (_rand(45 + i, 200, 2, 64, dtype=F16) for i in range(3))
    clean = _run_prompt(m, q, k, v, cu, cu, F16)
    k[150:], v[150, 0, 3], v[151, 1, 60], v[199] = float("nan"), float("nan"), float("inf"), float("-inf")
    got = _run_prompt(m, q, k, v, cu, cu, F16)
    assert torch.equal(clean[:150], got[:150]) and got[150:].isnan().all()


def test_prompt_values_that_are_not_finite_reach_who_sees_them(m):
    cu = _cu([300])
    q, k, v = (_rand(48 + i, 300, 2, 128, dtype=BF16) for i in range(3))
    clean = _run_prompt(m, q, k, v, cu, cu, BF16)
    v[210, 0, 5], v[280, 1, 100], v[290, 1, 100], v[220, 1, 7] = float("inf"), float("inf"), float("-inf"), float("nan")
    got = _run_prompt(m, q, k, v, cu, cu, BF16).cpu()
    want = clean.cpu().clone()
    want[210:, 0, 5], want[280:, 1, 100], want[290:, 1, 100], want[220:, 1, 7] = float("inf"), float("inf"), float("nan"), float("nan")
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~want.isnan()], want[~want.isnan()])


def test_prompt_peaked_logits_move_the_reference(m):
    cu = _cu([700])
    q, k, v = _rand(50, 700, 2, 128, dtype=F16, scale=2.5), _rand(51, 700, 2, 128, dtype=F16, scale=2.5), _rand(52, 700, 2, 128, dtype=F16)
    k *= torch.linspace(0.2, 2.0, 700)[:, None, None].half()
    _check_prompt(_run_prompt(m, q, k, v, cu, cu, F16, scale=0.5), q, k, v, cu, cu, F16, True, 0.5)


# Few queries before long keys: each unit's keys are cut over a cluster of 2, 4 or 8 CTAs.
CUT = [([1], [2000], 8, 1, 128, BF16, True), ([1], [4100], 8, 2, 64, F16, True), ([3, 0, 1], [1500, 700, 2600], 12, 4, 64, BF16, True),
       ([40, 1], [5000, 3], 6, 2, 128, F16, True), ([130], [4200], 1, 1, 128, BF16, False), ([64], [1100], 128, 1, 64, F16, True),
       ([600, 2], [40, 9000], 2, 2, 64, BF16, True), ([1, 1, 1], [0, 8000, 129], 32, 8, 128, BF16, True), ([33], [1500], 7, 1, 128, F16, False)]


@pytest.mark.parametrize("nq,nk,hq,hk,d,dtype,causal", CUT)
def test_prompt_few_queries_before_long_keys(m, nq, nk, hq, hk, d, dtype, causal):
    cu_q, cu_k = _cu(nq), _cu(nk)
    q, k, v = _rand(55, sum(nq), hq, d, dtype=dtype), _rand(56, sum(nk), hk, d, dtype=dtype), _rand(57, sum(nk), hk, d, dtype=dtype)
    got = _run_prompt(m, q, k, v, cu_q, cu_k, dtype, causal=causal, pad=8)
    _check_prompt(got, q, k, v, cu_q, cu_k, dtype, causal, None, str((nq, nk)))
    assert torch.equal(got, _run_prompt(m, q, k, v, cu_q, cu_k, dtype, causal=causal))


def test_prompt_cut_keys_hold_what_nobody_else_sees(m):
    """As for long prompts: infinities and NaN of V reach the queries that see them, across the cuts (each block of
    the first sequence's 300 keys is another CTA's), those of another sequence nobody."""
    cu_q, cu_k = _cu([200, 64, 3]), _cu([300, 9000, 2000])
    q, k, v = _rand(65, 267, 2, 128, dtype=BF16), _rand(66, 11300, 2, 128, dtype=BF16), _rand(67, 11300, 2, 128, dtype=BF16)
    clean = _run_prompt(m, q, k, v, cu_q, cu_k, BF16).cpu()
    v[210, 0, 5], v[280, 1, 100], v[290, 1, 100], v[220, 1, 7], v[127, 0, 9], v[128, 0, 10] = (
        float(x) for x in ("inf", "inf", "-inf", "nan", "-inf", "inf"))
    v[400, 0, 1] = float("inf")
    q[264:], k[9300:], v[9300:] = float("nan"), float("inf"), float("nan")
    got = _run_prompt(m, q, k, v, cu_q, cu_k, BF16).cpu()
    want = clean.clone()
    inf, nan = float("inf"), float("nan")
    want[110:200, 0, 5], want[180:200, 1, 100], want[190:200, 1, 100], want[120:200, 1, 7] = inf, inf, nan, nan
    want[27:200, 0, 9], want[28:200, 0, 10], want[200:264, 0, 1], want[264:] = -inf, inf, inf, nan
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~want.isnan()], want[~want.isnan()])


def test_prompt_cut_keys_with_peaked_logits(m):
    """The parts' references lie far apart, the largest logits in any of them."""
    size = torch.linspace(0.05, 2.0, 4000)[:, None, None].half()
    for sizes in (size, size.flip(0)):
        cu_q, cu_k = _cu([20]), _cu([4000])
        q, k, v = _rand(58, 20, 4, 64, dtype=F16, scale=2.5), _rand(59, 4000, 1, 64, dtype=F16, scale=2.5), _rand(60, 4000, 1, 64, dtype=F16)
        k *= sizes
        _check_prompt(_run_prompt(m, q, k, v, cu_q, cu_k, F16, scale=0.5), q, k, v, cu_q, cu_k, F16, True, 0.5)


# Enough units for two and more on every SM.
@pytest.mark.parametrize("nq,nk,hq,hk,d,dtype,causal", [
    ([130, 257, 1, 400], [130, 257, 1, 400], 48, 48, 64, F16, True), ([130, 257, 1, 400], [130, 300, 513, 400], 48, 48, 128, BF16, True),
    ([300, 700, 33], [300, 1000, 20], 63, 21, 64, BF16, True), ([500, 520, 9], [500, 520, 700], 128, 32, 128, F16, True),
    ([200, 300], [70, 513], 80, 80, 64, F16, False)])
def test_prompt_many_units(m, nq, nk, hq, hk, d, dtype, causal):
    cu_q, cu_k = _cu(nq), _cu(nk)
    q, k, v = _rand(120, sum(nq), hq, d, dtype=dtype), _rand(121, sum(nk), hk, d, dtype=dtype), _rand(122, sum(nk), hk, d, dtype=dtype)
    got = _run_prompt(m, q, k, v, cu_q, cu_k, dtype, causal=causal, pad=8)
    _check_prompt(got, q, k, v, cu_q, cu_k, dtype, causal, None, str((nq, nk)))
    assert torch.equal(got, _run_prompt(m, q, k, v, cu_q, cu_k, dtype, causal=causal))


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_many_units_values_that_are_not_finite(m, d):
    cu, h = _cu([300]), 160
    q, k, v = (_rand(125 + i, 300, h, d, dtype=BF16) for i in range(3))
    clean = _run_prompt(m, q, k, v, cu, cu, BF16).cpu()
    inf, nan = float("inf"), float("nan")
    v[210, 0, 5], v[280, 1, 60], v[290, 1, 60], v[220, 159, 7] = inf, inf, -inf, nan
    got = _run_prompt(m, q, k, v, cu, cu, BF16).cpu()
    want = clean.clone()
    want[210:, 0, 5], want[280:, 1, 60], want[290:, 1, 60], want[220:, 159, 7] = inf, inf, nan, nan
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~want.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("h,d", [(2, 64), (104, 64), (104, 128)])
def test_prompt_peaked_logits_in_each_kernel(m, h, d):
    """The reference moves in many blocks: sums that are being added to are multiplied."""
    cu = _cu([700])
    q, k, v = _rand(130, 700, h, d, dtype=F16, scale=2.5), _rand(131, 700, h, d, dtype=F16, scale=2.5), _rand(132, 700, h, d, dtype=F16)
    k *= torch.linspace(0.2, 2.0, 700)[:, None, None].half()
    _check_prompt(_run_prompt(m, q, k, v, cu, cu, F16, scale=0.5), q, k, v, cu, cu, F16, True, 0.5)


@pytest.mark.parametrize("nq,h", [(3, 1), (300, 40)])
def test_prompt_very_long_keys(m, nq, h):
    """Logits of size 8 over long keys: the largest weights, wherever they lie, make the result."""
    n, d = 150000 if h == 1 else 20000, 64
    cu_q, cu_k = _cu([nq]), _cu([n])
    q, k, v = _rand(140, nq, h, d, dtype=BF16), _rand(141, n, h, d, dtype=BF16), _rand(142, n, h, d, dtype=BF16)
    got = _run_prompt(m, q, k, v, cu_q, cu_k, BF16, scale=1.0)
    pick = [0, 1, nq - 1]  # (rows by themselves: a query sees the keys up to its own place)
    for i in pick:
        seen = n - nq + i + 1
        one, to = np.array([0, 1], dtype=np.int32), np.array([0, seen], dtype=np.int32)
        _check_prompt(got[i:i + 1], q[i:i + 1], k[:seen], v[:seen], one, to, BF16, True, 1.0, f"row {i}")


def test_prompt_repeats_bitwise_on_another_stream(m):
    lens = [300, 17, 555]
    cu, n = torch.from_numpy(_cu(lens)).cuda(), sum(lens)
    q, k, v = (_rand(60 + i, n, 8 if i == 0 else 2, 128, dtype=BF16).cuda() for i in range(3))
    op = m.PromptAttention(8, 2, 128)
    a, b = torch.empty_like(q), torch.empty_like(q)
    op.run(q, k, v, cu, cu, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        op.run(q, k, v, cu, cu, b, stream=side.cuda_stream)
    assert op.sync_status(side.cuda_stream) == m.GEMM_OK
    assert torch.equal(a, b)


@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_prompt_repeats_bitwise_whatever_a_cta_had_before(m, d, dtype):
    """Which units a CTA takes, and so which tile has a unit's first block, differs from run to run."""
    cu_q, cu_k = torch.from_numpy(_cu([1500, 1500, 995])).cuda(), torch.from_numpy(_cu([1503, 1501, 1000])).cuda()
    q, k, v = (_rand(150 + i, 3995 if i == 0 else 4004, 8 if i == 0 else 2, d, dtype=dtype).cuda() for i in range(3))
    op = m.PromptAttention(8, 2, d, dtype=m.GEMM_BF16 if dtype == BF16 else m.GEMM_F16)
    outs = [torch.empty_like(q) for _ in range(30)]
    for out in outs:
        op.run(q, k, v, cu_q, cu_k, out)
        torch.cuda.synchronize()
    assert op.sync_status() == m.GEMM_OK
    assert all(torch.equal(outs[0], out) for out in outs)


def test_prompt_refusals(m):
    op = m.PromptAttention(4, 2, 64, dtype=m.GEMM_F16)
    q, k = torch.zeros(5, 4, 64, dtype=torch.float16, device="cuda"), torch.zeros(6, 2, 64, dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.cpu()), dict(q=q[:, :2]), dict(q=q.bfloat16()), dict(v=k[:5]), dict(out=q[:4]), dict(cu_q=cu.long()),
                dict(cu_k=cu[:1]), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), dict(cu_q=cu[:0], cu_k=cu[:0])):
        with pytest.raises(ValueError):
            op.run(**{**dict(q=q, k=k, v=k, cu_q=cu, cu_k=cu, out=torch.empty_like(q)), **bad})
    with pytest.raises(TypeError):
        op.run(q, k, k, cu, cu, torch.empty_like(q), stream=torch.cuda.Stream())
    run, p = m._lib.attn_prompt_run, lambda t: t.data_ptr()
    ok = [op.plan, p(q), 0, p(k), 0, p(k), 0, p(cu), p(cu), 1, 5, 6, p(q), 0, None]
    for i, bad, st in ((0, None, 1), (1, None, 1), (3, None, 1), (5, None, 1), (7, None, 1), (8, None, 1), (12, None, 1), (9, -1, 1), (10, -1, 1),
                       (11, -1, 1), (2, 248, 1), (4, 132, 1), (6, 64, 1), (13, 260, 1), (1, p(q) + 8, 3), (7, p(cu) + 1, 3), (10, 1 << 31, 2)):
        assert run(*[bad if j == i else x for j, x in enumerate(ok)]) == st, (i, bad)
    assert run(*[0 if j == 9 else x for j, x in enumerate(ok)]) == m.GEMM_OK
    op.run(q[:0], k, k, cu * 0, cu, q[:0])


# ------------------------------------------------------------ the cache

@pytest.mark.parametrize("tokens,hk,d,page,dtype,pad", [(1, 1, 64, 16, F16, 0), (37, 3, 128, 48, BF16, 8), (500, 8, 128, 64, F16, 64),
                                                        (333, 5, 64, 1024, BF16, 0)])
def test_cache_codes_and_values_are_exact(m, tokens, hk, d, page, dtype, pad):
    pages = -(-tokens // page) + 2
    rng = np.random.default_rng(tokens)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    k, v = _rand(70, tokens, hk, d, dtype=dtype), _rand(71, tokens, hk, d, dtype=dtype)
    v *= torch.exp2(torch.from_numpy(rng.integers(-14 if dtype == F16 else -130, 14 if dtype == F16 else 120, (tokens, hk, 1))).float()).to(TD[dtype])
    if tokens > 8:
        k[0] = 0.0
        k[1, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0])
        k[2] = torch.finfo(TD[dtype]).max
        k[3] = torch.finfo(TD[dtype]).tiny * torch.finfo(TD[dtype]).eps  # the smallest subnormal
        k[4, 0] = float("nan")
    cache = m.KVCache.empty(pages, page, hk, d)
    ks, vs = _slices(tokens, hk, d, dtype, pad), _slices(tokens, hk, d, dtype, 0)
    ks.copy_(k), vs.copy_(v)
    cache.write(ks, vs, torch.from_numpy(slots).cuda())
    ko, vo = _slices(tokens, hk, d, dtype, 0), _slices(tokens, hk, d, dtype, pad)
    cache.read(torch.from_numpy(slots).cuda(), ko, vo)
    at, off = slots // page, slots % page
    for x, c, e, got in ((k, cache.k, cache.k_exp, ko), (v, cache.v, cache.v_exp, vo)):
        codes, exps = oracle.cache_encode(_val(x))
        nan = np.isnan(_val(x))
        assert np.array_equal(e.cpu().numpy()[at, :, off], exps)
        mine = c.cpu().numpy()[at, :, off]
        assert np.array_equal(np.where(nan, 127, mine & np.where(nan, 127, 255)), codes)
        want = np.clip(oracle.cache_decode(codes, exps), *(s * float(torch.finfo(TD[dtype]).max) for s in (-1, 1)))
        want = oracle.round_to(want, dtype)
        assert np.array_equal(_val(got), want, equal_nan=True)


def test_cache_leaves_out_slots_that_are_none(m):
    cache = m.KVCache.empty(2, 16, 2, 64)
    for t in (cache.k, cache.v, cache.k_exp, cache.v_exp):
        t.fill_(9)
    k, v = _rand(72, 4, 2, 64, dtype=F16).cuda(), _rand(73, 4, 2, 64, dtype=F16).cuda()
    slots = torch.tensor([-1, 32, 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    cache.write(k, v, slots)
    ko, vo = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    cache.read(slots, ko, vo)
    assert not ko[[0, 1, 3]].any() and not vo[[0, 1, 3]].any()
    assert ko[2].any() and (cache.k.flatten(0, 2)[: -17] == 9).all()
    assert int((cache.k_exp != 9).sum()) == 2
    cache.write(k[:0], v[:0], slots[:0])


def test_cache_refusals(m):
    cache = m.KVCache.empty(2, 16, 2, 64)
    k, slots = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for args in ((k.float(), k.float(), slots), (k, k[:3], slots), (k, k, slots.long()), (k, k, slots[:3]), (k[:, :1], k, slots),
                 (k, k.bfloat16(), slots), (k.cpu(), k, slots)):
        with pytest.raises(ValueError):
            cache.write(*args)
        with pytest.raises(ValueError):
            cache.read(args[2], args[0], args[1])
    with pytest.raises(m.GemmError):
        m.KVCache.empty(2, 24, 2, 64).write(k, k, slots)
    with pytest.raises(ValueError):
        m.KVCache(cache.k, cache.v, cache.k_exp, cache.v_exp[:1])


# ------------------------------------------------------------ attention over the cache

def _paged(m, lens, hk, d, page, seed, k_scale=1.0, v_power=None, spare=3):
    """A cache filled with random rows through its own write, a table of shuffled pages, and the fp64 values."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(max(need), 1)), -7, dtype=np.int32)
    used = 0
    for b, n in enumerate(need):
        table[b, :n] = order[used:used + n]
        used += n
    cache = m.KVCache.empty(pages, page, hk, d)
    # what no length covers: NaN codes and the largest exponents
    for t, fill in ((cache.k, 127), (cache.v, 255), (cache.k_exp, 254), (cache.v_exp, 254)):
        t.fill_(fill)
    ks, vs = [], []
    for b, n in enumerate(lens):
        if n == 0:
            ks.append(np.zeros((0, hk, d))), vs.append(np.zeros((0, hk, d)))
            continue
        k, v = _rand(seed + 2 * b, n, hk, d, dtype=BF16, scale=k_scale), _rand(seed + 2 * b + 1, n, hk, d, dtype=BF16)
        if v_power is not None:
            v = (v.float() * torch.from_numpy(2.0 ** rng.integers(*v_power, (n, hk, 1)))).bfloat16()
        at = np.arange(n)
        slots = torch.from_numpy((table[b][at // page] * page + at % page).astype(np.int32)).cuda()
        cache.write(k.cuda(), v.cuda(), slots)
        ks.append(oracle.cache_decode(*oracle.cache_encode(_val(k)))), vs.append(oracle.cache_decode(*oracle.cache_encode(_val(v))))
    return cache, table, ks, vs


def _check_decode(m, lens, hq, hk, d, page, dtype, seed=80, scale=0.0, q_scale=1.0, op=None, **kw):
    cache, table, ks, vs = _paged(m, lens, hk, d, page, seed, **kw)
    q = _rand(seed - 1, len(lens), hq, d, dtype=dtype, scale=q_scale)
    qs, out = _slices(len(lens), hq, d, dtype, 8), _slices(len(lens), hq, d, dtype, 16)
    qs.copy_(q)
    op = op or m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_BF16 if dtype == BF16 else m.GEMM_F16, scale=scale)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    op.run(qs, cache, torch.from_numpy(table).cuda(), n, out)
    s = scale or 1 / np.sqrt(d)
    for b, length in enumerate(lens):
        want, mag = oracle.prompt_attention(_val(q[b:b + 1]), ks[b], vs[b], [0, 1], [0, length], False, s)
        assert np.all(np.isfinite(_val(out[b]))), (lens, b)
        if length == 0:
            assert not out[b].any()
            continue
        big = np.sqrt((_val(q[b]) ** 2).sum(-1).max() * (ks[b] ** 2).sum(-1).max()) * s
        tol = _attention_tol(dtype, 2.0 ** -11, want, mag, (d + 4) * 2.0 ** -24 * big, length, np.abs(vs[b]).max(), extra=2.0 ** -24 * big)
        bad = np.abs(_val(out[b:b + 1]) - want) / np.maximum(tol, 1e-300)
        assert np.all(bad <= 1), f"{lens}, sequence {b}: {bad.max():.3g} of the tolerance"
    return op, cache, table, qs, n, out


@pytest.mark.parametrize("lens,hq,hk,d,page,dtype", [
    ([1], 1, 1, 64, 16, F16), ([0, 5, 0], 8, 2, 128, 64, BF16), ([15, 16, 17, 63, 64, 65, 127, 128, 129], 4, 1, 128, 16, F16),
    ([1000, 1, 300], 12, 2, 64, 48, BF16), ([5000], 8, 1, 128, 64, BF16), ([777, 20000], 8, 8, 64, 128, F16),
    ([40, 900], 16, 1, 128, 32, BF16), ([33, 2500], 30, 3, 64, 16, F16), ([600, 70], 40, 2, 128, 1024, F16), ([130], 64, 1, 64, 64, BF16)])
def test_decode_matches_oracle(m, lens, hq, hk, d, page, dtype):
    _check_decode(m, lens, hq, hk, d, page, dtype)


def test_decode_many_sequences(m):
    """More sequences than a block has threads; every run of tiles crosses several of them."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 150, 600)]
    _check_decode(m, lens, 4, 2, 64, 16, F16)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_rows_of_very_different_sizes(m, dtype):
    """Values' rows between 2^-20 and 2^8 of each other, peaked logits: the weights stay exact to the largest contribution."""
    _check_decode(m, [3000, 200], 4, 2, 128, 64, dtype, scale=0.5, q_scale=2.0, v_power=(-20, 6))


def test_decode_extreme_exponents(m):
    """bf16 values' rows anywhere in the type's range (results past fp16's range included)."""
    _check_decode(m, [500], 2, 1, 64, 16, BF16, v_power=(-100, 100))
    _check_decode(m, [500], 2, 1, 64, 16, BF16, q_scale=2.0 ** 60, k_scale=2.0 ** -60)


def test_decode_bad_pages_count_as_no_keys(m):
    lens, page = [160, 48], 16
    op, cache, table, q, n, out = _check_decode(m, lens, 4, 1, 64, page, F16)
    want = out.clone()
    hole = table.copy()
    hole[0, 2], hole[0, 5], hole[1, :] = -1, cache.pages, 2 ** 31 - 1
    op.run(q, cache, torch.from_numpy(hole).cuda(), n, out)
    assert not out[1].any() and torch.isfinite(out[0]).all() and not torch.equal(out[0], want[0])
    keep = [i for i in range(10) if i not in (2, 5)]
    short = np.full((2, 10), -1, dtype=np.int32)
    short[0, :8] = table[0, keep]
    n2 = torch.tensor([128, 0], dtype=torch.int32, device="cuda")
    dense = torch.empty_like(out)
    op.run(q, cache, torch.from_numpy(short).cuda(), n2, dense)
    assert torch.allclose(out[0].float(), dense[0].float(), rtol=2.0 ** -9, atol=2.0 ** -11)
    # a length past the table is cut to it
    n3 = torch.tensor([10 ** 6, -5], dtype=torch.int32, device="cuda")
    op.run(q, cache, torch.from_numpy(table).cuda(), n3, out)
    assert torch.equal(out[0], want[0]) and not out[1].any()


@pytest.mark.parametrize("lens,hq,hk,d,page,dtype", [
    ([169] * 20 + [0], 16, 8, 128, 48, BF16), ([50] * 100, 4, 4, 64, 16, F16), ([(7 * i) % 60 for i in range(90)], 12, 4, 128, 16, F16),
    ([257] * 31, 45, 5, 64, 64, BF16)])
def test_decode_more_short_passes_than_ctas(m, lens, hq, hk, d, page, dtype):
    """Whole ones to a CTA, one or several."""
    op, cache, table, q, n, out = _check_decode(m, lens, hq, hk, d, page, dtype)
    again = torch.empty_like(out)
    op.run(q, cache, torch.from_numpy(table).cuda(), n, again)
    assert torch.equal(out, again)


def test_decode_repeats_bitwise_and_grows(m):
    op, cache, table, q, n, out = _check_decode(m, [9000, 30, 4000], 8, 2, 128, 64, BF16)
    first, t = out.clone(), torch.from_numpy(table).cuda()
    for _ in range(20):
        op.run(q, cache, t, n, out)
        assert torch.equal(out, first)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert not op.workspace[-4 * (op.batch * 2 + 2 * sms):].any()  # the counters are zero again
    small = m.CacheAttention(8, 2, 128, 64, batch=1)
    again = torch.empty_like(first)
    small.run(q, cache, t, n, again)
    assert small.batch == 3 and torch.equal(again, first)


def test_decode_nan_in_a_seen_key_shows(m):
    op, cache, table, q, n, out = _check_decode(m, [100, 90], 4, 2, 64, 16, F16)
    want = out.clone()
    cache.k[table[0, 3], 1, 5, 7] = 127  # key 53 of sequence 0, key head 1
    op.run(q, cache, torch.from_numpy(table).cuda(), n, out)
    assert out[0, 2:].isnan().all() and torch.equal(out[0, :2], want[0, :2]) and torch.equal(out[1], want[1])


def test_decode_refusals(m):
    op, cache, table, q, n, out = _check_decode(m, [100, 90], 4, 2, 64, 16, F16)
    t = torch.from_numpy(table).cuda()
    for bad in (dict(q=q.cpu()), dict(q=q[:1]), dict(q=q.bfloat16()), dict(out=out[:1]), dict(lengths=n.long()), dict(lengths=n[:1]),
                dict(page_table=t.long()), dict(page_table=t[:1]), dict(page_table=t.t().contiguous().t()), dict(cache=m.KVCache.empty(4, 32, 2, 64))):
        with pytest.raises(ValueError):
            op.run(**{**dict(q=q, cache=cache, page_table=t, lengths=n, out=out), **bad})
    st = m._lib.attn_cache_attend(cache._ref, q.data_ptr(), q.stride(0), 4, t.data_ptr(), 0, t.shape[1], n.data_ptr(), 2, 0.0, m.GEMM_F16,
                                  out.data_ptr(), out.stride(0), op.workspace.data_ptr(), 64, None)
    assert st == m.GEMM_ERR_WORKSPACE
    op.run(q[:0], cache, t[:0], n[:0], out[:0])


# ------------------------------------------------------------ together

def test_one_layer_prompt_then_tokens(m):
    """A prompt through norm and rotation, cache and packed attention, then one more token over the cache: the
    token's result is that of a prompt one longer, up to the cache's rounding."""
    hq, hk, d, page, n = 8, 2, 128, 16, 150
    rope, prompt, decode = m.QKNormRope(hq, hk, d), m.PromptAttention(hq, hk, d), m.CacheAttention(hq, hk, d, page)
    qkv = _rand(90, n + 1, (hq + 2 * hk) * d, dtype=BF16).cuda()
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hk * d, hk * d], 1))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rope.run(q, k, torch.arange(n + 1, dtype=torch.int32, device="cuda"), q, k, w, w)
    cache = m.KVCache.empty(12, page, hk, d)
    order = torch.randperm(12, generator=torch.Generator().manual_seed(0)).int().cuda()
    at = torch.arange(n + 1, device="cuda")
    slots = order[at // page] * page + (at % page).int()
    cache.write(k, v, slots)
    ck, cv = torch.empty(n + 1, hk, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n + 1, hk, d, dtype=torch.bfloat16, device="cuda")
    cache.read(slots, ck, cv)
    cu = torch.tensor([0, n + 1], dtype=torch.int32, device="cuda")
    whole, token = torch.empty_like(q.contiguous()), torch.empty(1, hq, d, dtype=torch.bfloat16, device="cuda")
    prompt.run(q, ck, cv, cu, cu, whole)
    decode.run(q[n:], cache, order[None], torch.tensor([n + 1], dtype=torch.int32, device="cuda"), token)
    # both take the cache's values: they differ by the weights' and the results' rounding
    diff = (whole[n].float() - token[0].float()).abs()
    assert float(diff.max()) <= 4 * 2.0 ** -8 * float(cv.float().abs().max())


def test_cache_offsets_past_32_bits(m):
    """Pages whose codes lie past 2^32 bytes: written, read back and attended to there."""
    hq, hk, d, page, n = 8, 8, 128, 64, 200
    pages = (1 << 32) // (hk * page * d) + 8
    cache = m.KVCache.empty(pages, page, hk, d)
    table = torch.tensor([[pages - 1, 3, pages - 7, pages - 2]], dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    slots = table[0, at // page] * page + (at % page).int()
    k, v = _rand(100, n, hk, d, dtype=F16).cuda(), _rand(101, n, hk, d, dtype=F16).cuda()
    cache.write(k, v, slots)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.read(slots, ko, vo)
    for x, got in ((k, ko), (v, vo)):
        assert np.array_equal(_val(got), oracle.cache_decode(*oracle.cache_encode(_val(x))))
    q, out = _rand(102, 1, hq, d, dtype=F16).cuda(), torch.empty(1, hq, d, dtype=torch.float16, device="cuda")
    m.CacheAttention(hq, hk, d, page, dtype=m.GEMM_F16).run(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), out)
    want, mag = oracle.prompt_attention(_val(q), _val(ko), _val(vo), [0, 1], [0, n], False)
    tol = _attention_tol(F16, 2.0 ** -11, want, mag, (d + 5) * 2.0 ** -24 * 60, n, 8.0)
    assert np.all(np.abs(_val(out) - want) <= tol)


@pytest.mark.parametrize("hk", [1, 16, 80])
def test_prompt_offsets_past_32_bits(m, hk):
    """Rows 2^23 values apart, the last ones past 2^32: the result of the same rows side by side, for the units' keys
    cut over clusters, few units and many.  (An infinity among the last values is fetched by itself.)"""
    n, d, stride = 1000, 64, 1 << 23
    big = torch.empty((n - 1) * stride + 4 * hk * d, dtype=torch.float16, device="cuda")
    far = [big[i * hk * d:].as_strided((n, hk, d), (stride, d, 1)) for i in range(4)]
    near = [_rand(110 + i, n, hk, d, dtype=F16).cuda() for i in range(3)]
    near[2][n - 5, hk - 1, 3] = float("inf")
    near.append(torch.empty_like(near[0]))
    for x, y in zip(far[:3], near):
        x.copy_(y)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    op = m.PromptAttention(hk, hk, d, dtype=m.GEMM_F16)
    op.run(*near[:3], cu, cu, near[3])
    op.run(*far[:3], cu, cu, far[3])
    assert op.sync_status() == m.GEMM_OK
    assert torch.equal(near[3], far[3]) and near[3][n - 5:, hk - 1, 3].isposinf().all()


def test_rope_offsets_past_32_bits(m):
    """Rows 2^25 values apart: the last ones start past 2^31 values."""
    t, d, stride = 66, 64, 1 << 25
    big = torch.empty((t - 1) * stride + 2 * d, dtype=torch.float16, device="cuda")
    x = big.as_strided((t, 2, d), (stride, d, 1))
    q = _rand(103, t, 2, d, dtype=F16)
    x.copy_(q)
    k = torch.zeros(t, 1, d, dtype=torch.float16, device="cuda")
    pos = torch.arange(t, dtype=torch.int32) * 1000
    m.QKNormRope(2, 1, d, dtype=m.GEMM_F16).run(x, k, pos.cuda(), x, k)
    _check_rope(x, q, pos.numpy(), oracle.rope_frequencies(d, 10000.0), True, None, 0.0, 1.0, F16, "far rows")


def test_example_layer_serves_what_a_longer_prompt_gives(m):
    """The example's tokens over the cache against the same tokens as the last of longer prompts (whose keys and
    values are not rounded to 8 bits).  The outputs have rms of about 1 / sqrt(visible keys); e4m3 holds a value to
    2^-4, so an output to about a tenth of its rms, a quarter with room for the logits' share."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_layer.py")
    spec = importlib.util.spec_from_file_location("serving_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    prompts, hidden = (40, 3, 130), 256
    outs = ex.serve(prompts, new_tokens=1, hidden=hidden, q_heads=4, k_heads=2, head_dim=64, page_size=16)
    assert [tuple(o.shape) for o in outs] == [(173, hidden), (3, hidden)] and all(torch.isfinite(o).all() for o in outs)
    # the same layer and inputs, the new token appended to each prompt
    layer = ex.AttentionLayer(hidden, 4, 2, 64, 64, 16, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    torch.randperm(3 * 9, generator=g, device="cuda")
    x = torch.randn(sum(prompts), hidden, generator=g, device="cuda").bfloat16()
    new = torch.randn(3, hidden, generator=g, device="cuda").bfloat16()
    cu = np.cumsum([0, *prompts])
    longer = torch.cat([torch.cat([x[a:b], new[i:i + 1]]) for i, (a, b) in enumerate(zip(cu[:-1], cu[1:]))])
    position = torch.cat([torch.arange(p + 1) for p in prompts]).int().cuda()
    cu1 = torch.from_numpy((cu + np.arange(4)).astype(np.int32)).cuda()
    whole = layer.prompt(longer, position, torch.arange(176, dtype=torch.int32, device="cuda"), cu1)
    last = whole[(cu1[1:] - 1).long()].float()
    token = outs[1].float()
    assert float((token - last).norm() / last.norm()) < 0.25
    # and the prompts' own outputs do not depend on what follows them
    keep = torch.cat([torch.arange(p + 1) < p for p in prompts]).cuda()
    assert float((whole[keep].float() - outs[0].float()).norm() / outs[0].float().norm()) < 2.0 ** -7
