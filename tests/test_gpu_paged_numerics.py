"""How exact the paged attention is, token by token, against oracle/paged.py (binary64).

Where tests/test_gpu_paged.py allows every token the error of the batch's largest logit and value, these tests allow
each token its own, so that a token of large keys or values and little weight cannot blur the others unnoticed.

Tolerances, derived before any run.  Of token j with logit x, weight p (binary64) and value v:
- the logit is a sum of products in binary32 in any order, codes unsigned up to 15: off by 128 * 2^-23 of the sum of the
  products' magnitudes, delta; scaling it, adding the value scale's power of two (at most 2^7 in magnitude) and the
  reference round it three times more: 2^-22 (|x| + 130); the exponential is good to 2^-20;
- so the weight is off by eps = 2 delta + 2^-22 (|x| + |lse| + 130) + 2^-20 relative, and a weight that multiplies a value
  by half a step of its type besides: 2^-11 (4-bit rows, fp16), 2^-16 (bf16 rows, two bf16 parts);
- out is off by sum p (eps + step) |v| + |out| sum p eps, and by n 2^-23 sum p |v| for the binary32 accumulation;
- fp16 has an absolute floor, multiples of 2^-24: weights times a token's value scale are held in units in which the
  largest is at least 2^9, each off by at most 2^-34 of that largest, a code is at most 8: n 2^-31 of it over n tokens;
- a 4-bit value, and a key in calls of more than 32 rows, is a multiple of 2^-24 in units in which its token's largest
  scale is 2^-6 or more: exact where its own scale is at least 2^-11 of that largest, else off by 2^-19 of it ("apart").
Everything is checked on out_f32, before the last rounding.
"""
import numpy as np
import pytest

from oracle import paged as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import long_context_sparse_spa_b200 as spa  # noqa: E402
from test_gpu_paged import BF16, INT4, INVALID, Cache, _bf, _i32, _np  # noqa: E402


def put(c, b, n, k, v):
    """Token n of sequence b (one kv head) becomes k, v [d] fp32, in the pool and in the cache's binary64 copy."""
    k, v = np.asarray(k, np.float32)[None, None], np.asarray(v, np.float32)[None, None]
    at = (int(c.table[b, n // c.page]), slice(None), n % c.page)
    if c.fmt == INT4:
        row = ref.pack(k, v)
        c.pool[at] = torch.from_numpy(row[:, 0]).cuda()
        K, V, ks, vs = ref.unpack(row)
        c.ks[b][:, n], c.vs[b][:, n] = ks[:, 0], vs[:, 0]
    else:
        kb, vb = ref.bf16_bits(k), ref.bf16_bits(v)
        bits = np.stack((kb, vb), 2)[:, 0].astype(np.int32)
        c.pool.view(torch.int16)[at] = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).cuda()
        K, V = ref.bf16_value(kb).astype(np.float64), ref.bf16_value(vb).astype(np.float64)
    c.K[b][:, n], c.V[b][:, n] = K[:, 0], V[:, 0]


def check_closely(c, q, out, lse, sees, sm_scale, b, what, apart=False, floor=1e-40):
    """q [G, d], out [G, d] fp32 of one token and the one kv head, sees [n] bool."""
    K, V = c.K[b][0][sees], c.V[b][0][sees]
    n = len(K)
    for h in range(len(q)):
        o, z = ref.attend(q[h:h + 1], c.K[b][0], c.V[b][0], sees, sm_scale)
        o, z = o[0], z[0]
        x = K @ q[h] * sm_scale
        p = np.exp(x - z)
        per = np.repeat(c.ks[b][0][sees], c.d // 4, -1) * 15 if c.fmt == INT4 else np.abs(K)
        delta = sm_scale * (per * np.abs(q[h])).sum(-1) * 128 * 2.0**-23
        if apart:
            delta = delta + sm_scale * 2.0**-19 * c.ks[b][0][sees].max(-1) * np.abs(q[h]).sum()
        eps = 2 * delta + 2.0**-22 * (np.abs(x) + abs(z) + 130) + 2.0**-20
        off = (p * eps).sum()
        step = 2.0**-11 if c.fmt == INT4 else 2.0**-16
        tol = (p * (eps + step)) @ np.abs(V) + np.abs(o) * off + n * 2.0**-23 * (p @ np.abs(V))
        if c.fmt == INT4:
            tol = tol + n * 2.0**-31 * (p * c.vs[b][0][sees].max(-1)).max()
        if apart:
            tol = tol + 2.0**-19 * (p * c.vs[b][0][sees].max(-1)).sum()
        tol = tol * 1.01 + floor
        err = np.abs(out[h] - o)
        assert (err <= tol).all(), f"{what}, head {h}: out off by {(err / tol).max():.2f} of the tolerance"
        assert abs(lse[h] - z) <= off + 2.0**-21 * max(abs(z), 200), f"{what}, head {h}: lse {lse[h]} vs {z}"


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("new", [60, 5, 1])
@pytest.mark.parametrize("where", ["seventh", "one"])
@pytest.mark.parametrize("ke,ve", [(0, 10), (0, 12), (0, 16), (0, 20), (0, 24), (12, 0), (20, 0), (24, 24)])
def test_tokens_of_large_keys_or_values_and_little_weight(d, new, where, ke, ve):
    # all tokens but a few have keys and values around 1; the few 2^ke and 2^ve times those, with a weight of about e^-30
    # (or none at all, where the keys are large): tiles that all queries see, and one at the end that some do not
    L, scale = 400, 12.8 / d
    c = Cache([L], 1, d, 16, INT4, seed=61)
    rng = np.random.default_rng(ke * 100 + ve + new)
    for n in range(L):
        big = n % 7 == 3 if where == "seventh" else n == 40
        k = rng.standard_normal(d) * 0.3 - (2.4 * 2.0**ke if big else 0.0)
        put(c, 0, n, k, rng.standard_normal(d) * (2.0**ve if big else 1.0))
    q = torch.from_numpy((1 + 0.3 * rng.standard_normal((new, 4, d))).astype(np.float32)).cuda().to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=scale, seq_start=_i32([0, new]), want_f32=True, **c.kw)
    assert spa.read_device_status(plan.ws) == 0
    for i in sorted({0, new // 2, new - 1}):
        check_closely(c, _bf(q)[i], _np(plan.out_f32)[i].astype(np.float64), _np(plan.lse)[i].astype(np.float64),
                      np.arange(L) <= L - new + i, scale, 0, f"query {i}")


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("L,new", [(1, 1), (40, 1), (40, 2), (33, 5)])
def test_values_of_equal_tokens_come_back_exactly(d, L, new):
    # all tokens of a sequence are the same: weights are equal, in the units of the softmax a power of two, and the output
    # is the 4-bit value itself up to binary32 (the reference's and the logit's rounding, 2^-18, and the accumulation)
    B = 6
    c = Cache([L] * B, 1, d, 16, INT4, seed=62)
    rng = np.random.default_rng(62)
    for b in range(B):
        k, v = rng.standard_normal((2, d))
        v *= np.repeat(2.0 ** rng.integers(-9, 2, 4), d // 4)       # groups of different sizes, and of zeros
        v[: d // 4] *= b != 3
        for n in range(L):
            put(c, b, n, k, v)
    q = torch.randn(B * new, 4, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32(np.arange(B + 1) * new), want_f32=True, **c.kw)
    out = _np(plan.out_f32).astype(np.float64)
    for t in range(B * new):
        v = c.V[t // new][0, 0]
        err = np.abs(out[t] - v)
        assert (err <= np.abs(v) * (2.0**-18 + L * 2.0**-23)).all(), f"row {t}: off by {(err / np.abs(v).max()).max():.2e}"


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("new", [60, 5, 1])
@pytest.mark.parametrize("vs", [1e-22, 1e-30])
def test_tiny_values(fmt, new, vs):
    # bf16 rows: whatever the size.  4-bit rows: exact down to scales of 2^-81, below within 2^-89
    c = Cache([400], 1, 128, 16, fmt, seed=63, vscale=vs)
    q = torch.randn(new, 4, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, seq_start=_i32([0, new]), want_f32=True, **c.kw)
    for i in sorted({0, new // 2, new - 1}):
        check_closely(c, _bf(q)[i], _np(plan.out_f32)[i].astype(np.float64), _np(plan.lse)[i].astype(np.float64),
                      np.arange(400) <= 400 - new + i, 0.09, 0, f"query {i}",
                      floor=2.0**-89 if fmt == INT4 and vs < 1e-24 else 1e-40)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("new", [60, 5, 1])
@pytest.mark.parametrize("span", [9, 20])
def test_groups_of_a_token_that_lie_far_apart(d, new, span):
    c = Cache([400], 1, d, 16, INT4, seed=64)
    rng = np.random.default_rng(64)
    for n in range(400):
        far = 2.0 ** -rng.integers(0, span + 1, (2, 4))
        far[:, rng.integers(0, 4)] = 1
        k, v = rng.standard_normal((2, d)) * np.repeat(far, d // 4, -1)
        put(c, 0, n, k, v)
    q = torch.randn(new, 4, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32([0, new]), want_f32=True, **c.kw)
    for i in sorted({0, new // 2, new - 1}):
        check_closely(c, _bf(q)[i], _np(plan.out_f32)[i].astype(np.float64), _np(plan.lse)[i].astype(np.float64),
                      np.arange(400) <= 400 - new + i, 0.1, 0, f"query {i}", apart=span > 9)


@pytest.mark.parametrize("new", [60, 5, 1])
def test_far_scales_beside_a_missing_page_and_a_value_that_is_not_finite(new):
    L, d, scale = 400, 128, 0.1
    c = Cache([L], 1, d, 16, INT4, seed=65)
    rng = np.random.default_rng(65)
    for n in range(L):
        big = n % 7 == 3
        put(c, 0, n, rng.standard_normal(d) * 0.3 - 2.4 * big, rng.standard_normal(d) * (2.0**20 if big else 1.0))
    # token 10, that every query sees: group 2 of its value; tokens 48-63: no page
    host = c.pool.reshape(c.pool.shape[0], 1, 16, -1)
    host[int(c.table[0, 0]), 0, 10, d + 12:d + 14] = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device="cuda")
    c.kw["page_table"][0, 3] = -1
    q = torch.from_numpy((1 + 0.3 * rng.standard_normal((new, 4, d))).astype(np.float32)).cuda().to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=scale, seq_start=_i32([0, new]), want_f32=True, **c.kw)
    assert spa.read_device_status(plan.ws) == INVALID
    n = np.arange(L)
    c.V[0][:, :, 64:96] = 0
    for i in sorted({0, new // 2, new - 1}):
        out = _np(plan.out_f32)[i].astype(np.float64)
        assert np.isnan(out[:, 64:96]).all()
        out[:, 64:96] = 0
        check_closely(c, _bf(q)[i], out, _np(plan.lse)[i].astype(np.float64), (n <= L - new + i) & ((n < 48) | (n >= 64)),
                      scale, 0, f"query {i}")
