"""Paged KV cache on the GPU: append with rotation, gather and attention, against oracle/paged.py (binary64).

Tolerances, derived from the formats before any run:
- a bf16 output is within half a step (2^-8 of its value) of the exact one, plus the binary32 error of the
  rotation (three roundings and two of cos and sin: 4 * 2^-24 of |x| + |y|);
- a 4-bit value is within scale / 2 of the exact one (plus the same rotation error), its scale the exact
  amax / 7 rounded up to bf16 from a binary32 amax;
- attention: weights are off by 3 * 2^-11 (4-bit: the weight, the group's scale relative to its token's largest,
  and their product with the code are rounded to fp16 once each) or 2^-15 (bf16: hi + lo), logits by
  delta = 128 * 2^-23 of the sum of the products' magnitudes (binary32 accumulation in any order, codes
  unsigned up to 15), which scales weights by e^(2 delta); outputs by their final rounding.
"""
import numpy as np
import pytest

from oracle import paged as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import long_context_sparse_spa_b200 as spa  # noqa: E402
from long_context_sparse_spa_b200 import _abi  # noqa: E402

BF16, INT4 = spa.SPA_KV_BF16, spa.SPA_KV_INT4
INVALID, TIMEOUT = 1 << _abi.SPA_ERR_INVALID_ARG, 1 << _abi.SPA_ERR_TIMEOUT


def _np(t):
    return t.detach().cpu().numpy()


def _bf(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Cache:
    """A pool with shuffled pages, its table, and (optionally) random contents as rows [b][g, n, ...]."""

    def __init__(self, lens, Hkv, d, page, fmt, seed=0, fill=True, kscale=1.0, vscale=1.0, spare=2, extra=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.d, self.page, self.fmt = list(lens), Hkv, d, page, fmt
        width = max(1, -(-max([*lens, 1]) // page)) + extra
        P = len(lens) * width + spare
        self.table = rng.permutation(P)[:len(lens) * width].reshape(len(lens), width).astype(np.int32)
        self.pool = spa.paged_cache(P, Hkv, page, d, fmt)
        # what lies past the lengths must never matter: all ones is NaN in every bf16 it is read as
        self.pool.view(torch.uint8).fill_(255)
        self.K, self.V, self.ks, self.vs = [], [], [], []
        if fill:
            host = _np(self.pool.view(torch.uint8)).reshape(P, Hkv, page, -1)
            for b, L in enumerate(lens):
                k = (rng.standard_normal((Hkv, L, d)) * kscale).astype(np.float32)
                v = (rng.standard_normal((Hkv, L, d)) * vscale).astype(np.float32)
                if fmt == INT4:
                    rows = ref.pack(k, v)
                    k, v, ks, vs = ref.unpack(rows)
                    self.ks.append(ks)
                    self.vs.append(vs)
                else:
                    kb, vb = ref.bf16_bits(k), ref.bf16_bits(v)
                    rows = np.concatenate((kb, vb), -1).astype("<u2").view(np.uint8)
                    k, v = ref.bf16_value(kb).astype(np.float64), ref.bf16_value(vb).astype(np.float64)
                for n in range(L):
                    host[self.table[b, n // page], :, n % page] = rows[:, n]
                self.K.append(k)
                self.V.append(v)
            self.pool.view(torch.uint8).copy_(torch.from_numpy(host).reshape(self.pool.view(torch.uint8).shape))
        self.kw = dict(cache=self.pool, page_table=torch.from_numpy(self.table).cuda(), kv_len=_i32(lens))

    def row(self, pool, b, n):
        """Raw bytes [Hkv, row] of token n of sequence b."""
        P = pool.shape[0]
        return pool.reshape(P, self.Hkv, self.page, -1)[self.table[b, n // self.page], :, n % self.page]


def check_attention(c, q, out, lse, sees, sm_scale, b, what):
    """q [Hq, d] bf16 values of one token, sees [Hkv or Hq][n] bool."""
    Hq = len(q)
    G = Hq // c.Hkv
    for g in range(c.Hkv):
        for h in range(g * G, (g + 1) * G):
            s = sees[h] if len(sees) == Hq and len(sees) != c.Hkv else sees[g]
            o, z = ref.attend(q[h:h + 1], c.K[b][g], c.V[b][g], s, sm_scale)
            o, z = o[0], z[0]
            if not s.any():
                assert (out[h] == 0).all() and lse[h] == -np.inf, what
                continue
            Ks = c.K[b][g][s]
            if c.fmt == INT4:
                mag = (np.repeat(c.ks[b][g][s], c.d // 4, -1) * 15 * np.abs(q[h])).sum(-1).max()
            else:
                mag = (np.abs(Ks) * np.abs(q[h])).sum(-1).max()
            delta = sm_scale * mag * 128 * 2.0**-23 + 2.0**-20
            p = np.exp(Ks @ q[h] * sm_scale - z)
            av = p @ np.abs(c.V[b][g][s])
            tol = np.abs(o) * 2.0**-8 + (2 * delta + (3 * 2.0**-11 if c.fmt == INT4 else 2.0**-15)) * av * 1.01 + 1e-30
            if c.fmt == INT4:
                # fp16 has an absolute floor, multiples of 2^-24.  Weights P = p * (their token's largest value scale)
                # are held in units in which the largest is at least 2^9, so below the floor each is off by at most
                # 2^-25 / 2^9 = 2^-34 of that largest; a code is at most 8 in magnitude: n * 2^-31 of it over n
                # tokens.  A value relative to its token's largest scale is held times 2^-6 at least, so below the
                # floor it is off by 2^-25 * 2^6 = 2^-19 of that scale; a relative scale is held times 2^15 and is
                # off by 2^-40, times a code of at most 8.
                big = p * c.vs[b][g][s].max(-1)
                tol = tol + len(p) * 2.0**-31 * big.max() + (2.0**-19 + 2.0**-37) * big.sum()
            err = np.abs(out[h] - o)
            assert (err <= tol).all(), f"{what}: head {h}, out off by {(err / tol).max():.2f} of the tolerance"
            assert abs(lse[h] - z) <= delta + 2.0**-21 * max(abs(z), 32), f"{what}: head {h}, lse {lse[h]} vs {z}"


# ------------------------------------------------------------------------------------------------ append
APPENDS = [
    # d, page, Hkv, G, fmt, rot, interleaved, new tokens, earlier tokens
    (128, 16, 8, 4, INT4, 128, False, [1, 1, 1], [0, 15, 131071]),
    (128, 64, 2, 8, INT4, 64, True, [3, 0, 70, 1], [0, 5, 63, 1000]),
    (64, 32, 1, 1, INT4, 32, False, [33, 1], [31, 999_999]),
    (64, 16, 3, 2, INT4, 64, True, [17], [16]),
    (128, 128, 4, 2, BF16, 128, False, [5, 130], [127, 0]),
    (64, 16, 2, 3, BF16, 16, True, [1, 1, 2], [0, 7, 123_456]),
    (128, 16, 1, 4, BF16, 48, False, [40], [9]),
    (64, 1024, 2, 1, INT4, 0, False, [600], [700]),
]


@pytest.mark.parametrize("d,page,Hkv,G,fmt,rot,inter,new,old", APPENDS)
@pytest.mark.parametrize("where", ["place", "positions"])
def test_append(d, page, Hkv, G, fmt, rot, inter, new, old, where):
    rng = np.random.default_rng(d + page + rot)
    lens = [a + b for a, b in zip(new, old)]
    c = Cache([0] * len(lens), Hkv, d, page, fmt, fill=False)
    width = -(-max(lens) // page) + 1
    # only the pages that receive tokens need to exist: the others share one
    table = np.zeros((len(lens), width), np.int32)
    nxt = 1
    for b, (a, n) in enumerate(zip(old, new)):
        for i in range(a // page, -(-(a + n) // page) if n else a // page):
            table[b, i], nxt = nxt, nxt + 1
    pool = spa.paged_cache(nxt, Hkv, page, d, fmt)
    pool.view(torch.uint8).fill_(0xA5)
    c.table = table
    T, lead, tail = sum(new), 2, 3          # rows before the first and behind the last sequence
    start = np.concatenate(([0], np.cumsum(new))) + lead
    qkv = torch.from_numpy(rng.standard_normal((lead + T + tail, (G + 2) * Hkv, d)).astype(np.float32)) \
        .to(torch.bfloat16).cuda()
    q, k, v = qkv[:, :G * Hkv], qkv[:, G * Hkv:(G + 1) * Hkv], qkv[:, (G + 1) * Hkv:]
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    place = np.zeros(lead + T + tail, np.int64)
    for b in range(len(lens)):
        place[start[b]:start[b + 1]] = np.arange(old[b], lens[b])
    pos = rng.integers(0, 1 << 20, len(place)) if where == "positions" else place
    q_out = torch.full((lead + T + tail, G * Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = spa.paged_append(k=k, v=v, q=q, q_out=q_out, cache=pool, page_table=torch.from_numpy(table).cuda(),
                            kv_len=_i32(lens), seq_start=_i32(start),
                            inv_freq=torch.from_numpy(inv).cuda() if rot else None, interleaved=inter,
                            positions=_i32(pos) if where == "positions" else None)
    assert spa.read_device_status(plan.ws) == 0
    got = _bf(q_out)
    want, raw = ref.rotate(_bf(q), pos, inv, inter), np.abs(_bf(q))
    slack = 8 * 2.0**-24 * raw.max()
    live = slice(lead, lead + T)
    assert (np.abs(got - want)[live] <= 2.0**-8 * np.abs(want[live]) + slack).all()
    assert (got[:lead] == 7).all() and (got[lead + T:] == 7).all()
    wk, wv = ref.rotate(_bf(k), pos, inv, inter), _bf(v)
    host = _np(pool.view(torch.uint8)).reshape(nxt, Hkv, page, -1)
    touched = np.zeros(host.shape[:3], bool)
    for b in range(len(lens)):
        for t in range(start[b], start[b + 1]):
            n = int(place[t])
            pg = table[b, n // page]
            touched[pg, :, n % page] = True
            row = host[pg, :, n % page]
            if fmt == BF16:
                y = ref.bf16_value(row.reshape(Hkv, 2 * d, 2).copy().view("<u2")[..., 0]).astype(np.float64)
                assert (np.abs(y[:, :d] - wk[t]) <= 2.0**-8 * np.abs(wk[t]) + slack).all()
                assert (y[:, d:] == wv[t]).all()
            else:
                K, V, ks, vs = ref.unpack(row)
                for y, s, z, sl in ((K, ks, wk[t], slack), (V, vs, wv[t], 0.0)):
                    top = np.abs(z.reshape(Hkv, 4, d // 4)).max(-1)
                    assert (s >= (top - sl) / 7 * (1 - 2.0**-23)).all()
                    assert (s <= (top + sl) / 7 * (1 + 2.0**-7 + 2.0**-22)).all()
                    sr = np.repeat(s, d // 4, -1)
                    assert (np.abs(y - z) <= sr / 2 * (1 + 2.0**-20) + sl).all()
                assert (row[:, d // 2:d] == ref.pack(wk[t].astype(np.float32), wv[t].astype(np.float32))[:, d // 2:d]).all()
    assert (host[~touched] == 0xA5).all()


def test_append_one_token_per_sequence_and_without_queries():
    c = Cache([1, 40, 17], 2, 128, 16, INT4, fill=False)
    k = torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_append(k=k, v=k, **c.kw)
    assert plan.q_out is None and spa.read_device_status(plan.ws) == 0
    host = _np(c.pool)
    for b, L in enumerate(c.lens):
        want = ref.pack(_bf(k[b]).astype(np.float32), _bf(k[b]).astype(np.float32))
        assert (c.row(host, b, L - 1) == want).all()


def test_append_poisons_groups_that_are_not_finite():
    d = 128
    c = Cache([4], 1, d, 16, INT4, fill=False)
    k = torch.randn(4, 1, d, device="cuda").to(torch.bfloat16)
    v = torch.randn(4, 1, d, device="cuda").to(torch.bfloat16)
    k[0, 0, 5], v[1, 0, 40], v[2, 0, :] = float("nan"), float("-inf"), 0
    k[3, 0, :] = 3e38                       # amax / 7 stays finite: the largest values still quantise
    spa.paged_append(k=k, v=v, seq_start=_i32([0, 4]), **c.kw)
    K, V, ks, vs = ref.unpack(np.stack([c.row(_np(c.pool), 0, n)[0] for n in range(4)]))
    assert np.isnan(K[0, :32]).all() and np.isfinite(K[0, 32:]).all()
    assert np.isnan(V[1, 32:64]).all() and np.isfinite(V[1, :32]).all() and np.isfinite(V[1, 64:]).all()
    assert (V[2] == 0).all() and (vs[2] == 0).all()
    assert (np.abs(K[3] - float(k[3, 0, 0])) <= ks[3].repeat(32) / 2 * 1.001).all()


def test_bad_pages_and_lengths_are_reported_and_not_written():
    for fmt in (INT4, BF16):
        c = Cache([20, 20, 20, 20], 2, 64, 16, fmt, fill=False)
        before = c.pool.clone()
        c.kw["page_table"][0, 1] = c.pool.shape[0]
        c.kw["page_table"][1, 1] = -5
        c.kw["kv_len"][2] = 10_000
        c.kw["kv_len"][3] = 0                # its one token would be token -1
        k = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
        q_out = torch.full_like(k, 3)
        plan = spa.paged_append(k=k, v=k, q=k, q_out=q_out, **c.kw)
        assert spa.read_device_status(plan.ws) == INVALID and spa.read_device_status(plan.ws) == 0
        assert torch.equal(c.pool.view(torch.uint8), before.view(torch.uint8)) and (q_out == 3).all()


# ------------------------------------------------------------------------------------------------ gather
@pytest.mark.parametrize("d,page,Hkv,fmt", [(128, 16, 3, INT4), (64, 64, 2, INT4), (128, 32, 1, BF16), (64, 16, 4, BF16)])
def test_gather(d, page, Hkv, fmt):
    c = Cache([0, 1, 63, 200], Hkv, d, page, fmt, seed=d)
    for start in (None, [0, 0, 40, 150]):
        N = 70
        K = torch.full((4, Hkv, N, d), 5.0, dtype=torch.bfloat16, device="cuda")
        V = torch.full_like(K, 5.0)
        plan = spa.paged_gather(N=N, start=None if start is None else _i32(start), K=K, V=V, **c.kw)
        assert spa.read_device_status(plan.ws) == 0
        for got, want in ((_bf(K), c.K), (_bf(V), c.V)):
            for b, L in enumerate(c.lens):
                s = start[b] if start else 0
                n = max(0, min(N, L - s))
                w = ref.bf16_value(ref.bf16_bits(want[b][:, s:s + n])).astype(np.float64)
                assert (got[b, :, :n] == w).all() and (got[b, :, n:] == 5).all()


def test_gather_skips_bad_pages():
    c = Cache([40, 40], 2, 64, 16, INT4, seed=3)
    c.kw["page_table"][0, 1] = 1 << 30
    plan = spa.paged_gather(N=48, start=_i32([0, -4]), **c.kw)
    assert spa.read_device_status(plan.ws) == INVALID
    K = _bf(plan.K)
    assert (K[0, :, 16:32] == 0).all() and (K[0, :, :16] != 0).any() and (K[1, :, :4] == 0).all()
    w = ref.bf16_value(ref.bf16_bits(c.K[1])).astype(np.float64)
    assert (K[1, :, 4:44] == w).all() and (K[:, :, 44:] == 0).all()


def test_gather_reads_pages_past_4_gib():
    P = 40_000                               # 40 000 pages x 8 heads x 128 tokens x 144 bytes = 5.9 GB
    pool = spa.paged_cache(P, 8, 128, 128, INT4)
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 8, 128, 128)).astype(np.float32)
    pool[P - 1].copy_(torch.from_numpy(ref.pack(k, v)))
    kw = dict(cache=pool, page_table=_i32([[P - 1]]), kv_len=_i32([128]))
    got = spa.paged_gather(N=128, **kw)
    K, V, _, _ = ref.unpack(ref.pack(k, v))
    assert (_bf(got.K)[0] == ref.bf16_value(ref.bf16_bits(K))).all()
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    a = spa.paged_attend(q=q, sm_scale=0.1, **kw)
    for g in range(8):
        o, _ = ref.attend(_bf(q)[0, g:g + 1], K[g], V[g], np.ones(128, bool), 0.1)
        assert np.abs(_bf(a.out)[0, g] - o[0]).max() <= 2.0**-7 * np.abs(V[g]).max()
    row = spa.paged_append(k=q, v=q, **{**kw, "kv_len": _i32([100])})
    assert spa.read_device_status(row.ws) == 0
    assert (_np(pool[P - 1, :, 99]) == ref.pack(_bf(q)[0].astype(np.float32), _bf(q)[0].astype(np.float32))).all()


# ------------------------------------------------------------------------------------------------ attention
LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200, 1001, 3000]


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("d,Hkv,G,page", [(128, 2, 8, 16), (128, 1, 4, 64), (64, 1, 4, 16), (64, 2, 1, 128), (128, 2, 3, 32),
                                          (64, 1, 16, 64), (128, 1, 16, 16), (128, 3, 6, 1024)])
def test_attend_one_query_per_sequence(fmt, d, Hkv, G, page):
    c = Cache(LENS, Hkv, d, page, fmt, seed=d + G)
    q = torch.randn(len(LENS), G * Hkv, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=d**-0.5, want_f32=True, **c.kw)
    assert spa.read_device_status(plan.ws) == 0
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    assert torch.equal(plan.out_f32.to(torch.bfloat16), plan.out)
    for b, L in enumerate(LENS):
        check_attention(c, qv[b], out[b], lse[b], [np.ones(L, bool)] * Hkv, d**-0.5, b, f"length {L}")


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("d,Hkv,G,page,new", [(128, 2, 4, 16, [1, 5, 0, 33, 2]), (64, 1, 8, 32, [7, 1, 16, 3, 0]),
                                              (128, 1, 16, 64, [2, 3, 1, 0, 4]), (64, 2, 3, 16, [11, 1, 40, 6, 5]),
                                              (128, 1, 1, 16, [20, 17, 64, 1, 9])])
def test_attend_several_queries_per_sequence(fmt, d, Hkv, G, page, new):
    lens = [1, 300, 40, 33, 1500]           # the second to last: its queries are the whole sequence
    new = [min(n, L) for n, L in zip(new, lens)]
    c = Cache(lens, Hkv, d, page, fmt, seed=G)
    lead, tail = 1, 2
    start = np.concatenate(([0], np.cumsum(new))) + lead
    T = lead + sum(new) + tail
    # queries as a slice of a fused projection: strides other than dense
    q = torch.randn(T, G * Hkv + 2, d, device="cuda").to(torch.bfloat16)[:, 1:-1]
    kw = dict(q=q, sm_scale=0.11, seq_start=_i32(start), want_f32=True, **c.kw)
    plan = spa.paged_attend(run=False, **kw)
    plan.out.fill_(9)
    plan.lse.fill_(9)
    plan.run()
    assert spa.read_device_status(plan.ws) == 0
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    assert (out[:lead] == 9).all() and (out[T - tail:] == 9).all() and (lse[T - tail:] == 9).all()
    for b, (n, L) in enumerate(zip(new, lens)):
        for i in range(n):
            sees = np.arange(L) <= L - n + i
            t = start[b] + i
            check_attention(c, qv[t], out[t], lse[t], [sees] * Hkv, 0.11, b, f"sequence {b}, query {i}")


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("d,Hkv,G,page,new,lens", [
    (128, 2, 4, 64, [200, 3, 0, 64], [1500, 700, 90, 64]),      # several row tiles, a whole prompt, one short
    (64, 1, 8, 16, [131], [131]),                               # a prompt from nothing
    (128, 1, 1, 128, [300, 1], [2111, 1]),                      # one head: 256 tokens to a unit
    (128, 3, 5, 16, [60, 52, 7], [60, 333, 4000]),              # rows that do not divide a tile
    (64, 2, 16, 32, [33, 20], [500, 129])])
def test_attend_a_chunk(fmt, d, Hkv, G, page, new, lens):
    c = Cache(lens, Hkv, d, page, fmt, seed=d + G + 1)
    start = np.concatenate(([0], np.cumsum(new)))
    q = torch.randn(int(start[-1]), G * Hkv, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=1.5 * d**-0.5, seq_start=_i32(start), want_f32=True, **c.kw)
    assert spa.read_device_status(plan.ws) == 0
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    assert torch.equal(plan.out_f32.to(torch.bfloat16), plan.out)
    rng = np.random.default_rng(G)
    for b, (n, L) in enumerate(zip(new, lens)):
        for i in sorted({0, 1, n // 2, n - 2, n - 1, *rng.integers(0, max(n, 1), 12)} & set(range(n))):
            t = start[b] + i
            check_attention(c, qv[t], out[t], lse[t], [np.arange(L) <= L - n + i] * Hkv, 1.5 * d**-0.5, b,
                            f"sequence {b}, query {i}")
    first = plan.out.clone()
    plan.run()
    assert torch.equal(first, plan.out)


def test_units_of_one_and_two_row_tiles_in_turn():
    # a CTA takes units of up to 128 rows and of more in turn, more of them than there are SMs: the second row tile's
    # warps sit out some units and must neither lag nor run ahead
    rng = np.random.default_rng(51)
    new = [int(x) for x in rng.choice([3, 20, 40, 64, 33, 50], 180)]
    lens = [int(n + x) for n, x in zip(new, rng.integers(0, 700, 180))]
    c = Cache(lens, 2, 128, 16, INT4, seed=51)
    start = np.concatenate(([0], np.cumsum(new)))
    q = torch.randn(int(start[-1]), 8, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, seq_start=_i32(start), **c.kw)
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    assert np.isfinite(out).all()
    for b in range(0, 180, 7):
        for i in (0, new[b] // 2, new[b] - 1):
            t = start[b] + i
            check_attention(c, qv[t], out[t], lse[t], [np.arange(lens[b]) <= lens[b] - new[b] + i] * 2, 0.09, b,
                            f"sequence {b}, query {i}")
    first = plan.out.clone()
    for _ in range(20):
        plan.run()
        assert torch.equal(first, plan.out)
    assert spa.read_device_status(plan.ws) == 0


def test_a_long_chunk_is_split_and_merged():
    c = Cache([30_000, 17], 1, 128, 64, INT4, seed=31)
    start = [0, 90, 107]
    q = (2 * torch.randn(107, 4, 128, device="cuda")).to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32(start), **c.kw)
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    for t in (0, 1, 31, 32, 63, 64, 88, 89, 90, 106):
        b, n = (0, 90) if t < 90 else (1, 17)
        L = c.lens[b]
        check_attention(c, qv[t], out[t], lse[t], [np.arange(L) <= L - n + t - start[b]], 0.1, b, f"row {t}")
    first = plan.out.clone()
    for _ in range(3):
        plan.run()
        assert torch.equal(first, plan.out)
    assert spa.read_device_status(plan.ws) == 0


@pytest.mark.parametrize("qs,ks,vs", [(1, 1, 1e-20), (1, 1, 1e30), (1e-20, 1e20, 1), (1e15, 1e-15, 1e-6), (40, 1, 1)])
def test_chunk_scales_far_from_one(qs, ks, vs):
    c = Cache([400], 1, 128, 16, INT4, seed=32, kscale=ks, vscale=vs)
    q = (qs * torch.randn(60, 4, 128, device="cuda")).to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, seq_start=_i32([0, 60]), **c.kw)
    for t in (0, 33, 59):
        check_attention(c, _bf(q)[t], _bf(plan.out)[t], _np(plan.lse)[t].astype(np.float64), [np.arange(400) <= 340 + t],
                        0.09, 0, f"row {t}")


def test_chunk_masks_what_is_not_finite_and_bad_pages():
    c = Cache([300], 1, 128, 16, INT4, seed=33)
    host = c.pool.reshape(c.pool.shape[0], 1, 16, -1)
    # token 260: its value's group 2 is NaN; token 290: its key; tokens 64-79: no page
    host[c.table[0, 16], 0, 4, 128 + 12:128 + 14] = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device="cuda")
    host[c.table[0, 18], 0, 2, 128:130] = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device="cuda")
    c.kw["page_table"][0, 4] = -3
    q = torch.randn(60, 4, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, seq_start=_i32([0, 60]), **c.kw)
    assert spa.read_device_status(plan.ws) == INVALID
    out, lse, n = _bf(plan.out), _np(plan.lse).astype(np.float64), np.arange(300)
    for t in (0, 10, 19, 20, 40, 49, 50, 59):
        sees = (n <= 240 + t) & ((n < 64) | (n >= 80))
        if t >= 50:
            assert np.isnan(out[t]).all() and np.isnan(lse[t]).all()
            continue
        o = out[t].copy()
        if t >= 20:
            assert np.isnan(o[:, 64:96]).all()
            o[:, 64:96] = 0
            c.V[0][:, 260, 64:96] = 0
            keep = c.V[0].copy()
            c.V[0][:, :, 64:96] = 0
            check_attention(c, _bf(q)[t], o, lse[t], [sees], 0.09, 0, f"row {t}")
            c.V[0] = keep
        else:
            check_attention(c, _bf(q)[t], o, lse[t], [sees], 0.09, 0, f"row {t}")


def test_bf16_units_of_one_and_two_row_tiles_in_turn():
    rng = np.random.default_rng(53)
    new = [int(x) for x in rng.choice([3, 20, 40, 64, 33, 50], 180)]
    lens = [int(n + x) for n, x in zip(new, rng.integers(0, 700, 180))]
    c = Cache(lens, 2, 64, 32, BF16, seed=53)
    start = np.concatenate(([0], np.cumsum(new)))
    q = torch.randn(int(start[-1]), 8, 64, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.15, seq_start=_i32(start), **c.kw)
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    for b in range(0, 180, 7):
        for i in (0, new[b] // 2, new[b] - 1):
            t = start[b] + i
            check_attention(c, qv[t], out[t], lse[t], [np.arange(lens[b]) <= lens[b] - new[b] + i] * 2, 0.15, b,
                            f"sequence {b}, query {i}")
    first = plan.out.clone()
    for _ in range(20):
        plan.run()
        assert torch.equal(first, plan.out)
    assert spa.read_device_status(plan.ws) == 0


@pytest.mark.parametrize("qs,ks,vs", [(1, 1, 1e-30), (1, 1, 1e30), (1e-20, 1e20, 1), (1e15, 1e-15, 1e-6), (40, 1, 1)])
def test_bf16_chunk_scales_far_from_one(qs, ks, vs):
    c = Cache([400], 1, 128, 16, BF16, seed=54, kscale=ks, vscale=vs)
    q = (qs * torch.randn(60, 4, 128, device="cuda")).to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, seq_start=_i32([0, 60]), **c.kw)
    for t in (0, 33, 59):
        check_attention(c, _bf(q)[t], _bf(plan.out)[t], _np(plan.lse)[t].astype(np.float64), [np.arange(400) <= 340 + t],
                        0.09, 0, f"row {t}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [300, 20_000])     # the longer one is split, and its shares merged
def test_bf16_chunk_masks_what_is_not_finite_and_bad_pages(d, L):
    c = Cache([L], 1, d, 16, BF16, seed=55)
    pool = c.pool
    hit = np.zeros(d, bool)
    hit[[0, 5, d - 1]] = True
    # token L - 40: its value in three channels; token L - 10: its key; tokens 64-79: no page
    n1, n2 = L - 40, L - 10
    for ch, x in zip(np.flatnonzero(hit), (np.nan, np.inf, -np.inf)):
        pool[int(c.table[0, n1 // 16]), 0, n1 % 16, 1, int(ch)] = float(x)
    pool[int(c.table[0, n2 // 16]), 0, n2 % 16, 0, 7] = float("nan")
    c.kw["page_table"][0, 4] = 1 << 30
    q = torch.randn(60, 4, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, seq_start=_i32([0, 60]), **c.kw)
    assert spa.read_device_status(plan.ws) == INVALID
    out, lse, n = _bf(plan.out), _np(plan.lse).astype(np.float64), np.arange(L)
    for t in (0, 10, 19, 20, 40, 49, 50, 59):
        sees = (n <= L - 60 + t) & ((n < 64) | (n >= 80))
        if t >= 50:
            assert np.isnan(out[t]).all() and np.isnan(lse[t]).all()
            continue
        o = out[t].copy()
        if t >= 20:
            assert not np.isfinite(o[:, hit]).any() and np.isfinite(o[:, ~hit]).all()
            o[:, hit] = 0
            keep = c.V[0].copy()
            c.V[0][:, :, hit] = 0
            check_attention(c, _bf(q)[t], o, lse[t], [sees], 0.09, 0, f"row {t}")
            c.V[0] = keep
        else:
            check_attention(c, _bf(q)[t], o, lse[t], [sees], 0.09, 0, f"row {t}")


def test_bf16_chunks_on_two_streams():
    cs = [Cache([700, 90, 300], 2, d, 16, BF16, seed=s, extra=2) for s, d in ((56, 128), (57, 64))]
    start = [0, 60, 61, 161]
    qs = [torch.randn(161, 8, c.d, device="cuda").to(torch.bfloat16) for c in cs]
    plans = [spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32(start), run=False, **c.kw) for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip(plans, streams):
            p.run(s)
    torch.cuda.synchronize()
    for c, q, p in zip(cs, qs, plans):
        assert spa.read_device_status(p.ws) == 0
        for b, L in enumerate([700, 90, 300]):
            n = start[b + 1] - start[b]
            for i in (0, n - 1):
                t = start[b] + i
                check_attention(c, _bf(q)[t], _bf(p.out)[t], _np(p.lse)[t].astype(np.float64),
                                [np.arange(L) <= L - n + i] * 2, 0.1, b, f"row {t}")


def test_queries_before_the_first_token_see_nothing():
    c = Cache([3], 1, 128, 16, INT4, seed=1)
    q = torch.randn(5, 4, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32([0, 5]), **c.kw)
    out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
    for i in range(5):
        check_attention(c, _bf(q)[i], out[i], lse[i], [np.arange(3) <= i - 2], 0.1, 0, f"query {i}")


@pytest.mark.parametrize("fmt", [INT4, BF16])
def test_a_long_sequence_is_split_and_merged(fmt):
    # one kv head over all SMs, and lengths that leave ragged shares
    for L in (20_011, 70_000):
        c = Cache([L], 1, 128, 64, fmt, seed=L)
        q = (3 * torch.randn(1, 8, 128, device="cuda")).to(torch.bfloat16)
        plan = spa.paged_attend(q=q, sm_scale=128**-0.5, **c.kw)
        assert spa.read_device_status(plan.ws) == 0
        check_attention(c, _bf(q)[0], _bf(plan.out)[0], _np(plan.lse)[0].astype(np.float64), [np.ones(L, bool)],
                        128**-0.5, 0, f"length {L}")
        first = plan.out.clone()
        for _ in range(3):                  # merged in a fixed order: equal calls give equal bits
            plan.run()
            assert torch.equal(first, plan.out)


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("collapse", [spa.SPA_COLLAPSE_GROUP_MEAN, spa.SPA_COLLAPSE_NONE])
@pytest.mark.parametrize("unit,page,d", [(1, 16, 128), (16, 64, 64), (64, 16, 128), (24, 32, 128), (3, 16, 64)])
def test_attend_supports(fmt, collapse, unit, page, d):
    Hkv, G = 2, 4
    lens = [0, 1, 500, 777, 2000]
    c = Cache(lens, Hkv, d, page, fmt, seed=unit)
    rng = np.random.default_rng(unit)
    per = Hkv if collapse == spa.SPA_COLLAPSE_GROUP_MEAN else Hkv * G
    U, cap = len(lens) * per, 45
    idx, count = np.full((U, cap), -7, np.int32), np.zeros(U, np.int32)
    sees = []
    for u in range(U):
        L = lens[u // per]
        M = -(-L // unit)
        k = min(M, int(rng.integers(0, cap + 1)))
        pick = np.sort(rng.permutation(M)[:k])
        idx[u, :k], count[u] = pick, k
        if u == U - 1 and k < cap:           # entries that name nothing: behind the sequence, and negative
            idx[u, k], count[u] = M + 3, k + 1
        s = np.zeros(L, bool)
        for e in pick:
            s[e * unit:(e + 1) * unit] = True
        sees.append(s)
    if U > 3:
        count[0] = -2                        # a negative count is an empty support
    q = torch.randn(len(lens), G * Hkv, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, idx=_i32(idx), count=_i32(count), collapse=collapse, unit_tokens=unit,
                            **c.kw)
    assert spa.read_device_status(plan.ws) == 0
    out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
    for b in range(len(lens)):
        s = [x & (lens[b] > 0) for x in sees[b * per:(b + 1) * per]]
        check_attention(c, _bf(q)[b], out[b], lse[b], s, 0.1, b, f"length {lens[b]}")


def test_supports_of_a_batch_with_empty_places():
    # sequences 1 and 3 have no query, sequence 4 (against the rules) two; rows of nobody stay
    Hkv, G, lens = 2, 2, [40, 30, 50, 0, 20]
    c = Cache(lens, Hkv, 64, 16, INT4, seed=21)
    q = torch.randn(5, Hkv * G, 64, device="cuda").to(torch.bfloat16)
    idx = np.tile(np.arange(6, dtype=np.int32), (5 * Hkv, 1))
    kw = dict(q=q, sm_scale=0.1, idx=_i32(idx), count=_i32(np.full(5 * Hkv, 6)), unit_tokens=4, **c.kw)
    for last, status in ((2, 0), (4, INVALID)):
        plan = spa.paged_attend(seq_start=_i32([0, 1, 1, 2, 2, last]), run=False, **kw)
        plan.out.fill_(9)
        plan.run()
        assert spa.read_device_status(plan.ws) == status
        out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
        for row, b in ((0, 0), (1, 2)):
            check_attention(c, _bf(q)[row], out[row], lse[row], [np.arange(lens[b]) < 24] * Hkv, 0.1, b, f"row {row}")
        assert (out[2:] == 9).all()


def test_count_above_cap_is_cut():
    c = Cache([100], 1, 128, 16, INT4, seed=2)
    q = torch.randn(1, 4, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, idx=_i32([[3, 9, 50]]), count=_i32([1 << 30]), **c.kw)
    s = np.zeros(100, bool)
    s[[3, 9, 50]] = True
    check_attention(c, _bf(q)[0], _bf(plan.out)[0], _np(plan.lse)[0].astype(np.float64), [s], 0.1, 0, "cut")


@pytest.mark.parametrize("fmt", [INT4, BF16])
def test_what_is_masked_does_not_matter(fmt):
    # the tokens after a query's own hold NaN and infinity: only the queries that see them may notice
    c = Cache([50], 1, 128, 16, fmt, seed=4)
    host = c.pool.view(torch.uint8).reshape(c.pool.shape[0], 1, 16, -1)
    for n, byte in ((47, 0xFF), (48, 0x7F), (49, 0xFF)):
        host[c.table[0, n // 16], 0, n % 16, 128 if fmt == INT4 else 0:].fill_(byte)
    q = torch.randn(6, 8, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32([0, 6]), **c.kw)
    out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
    for i in range(3):
        check_attention(c, _bf(q)[i], out[i], lse[i], [np.arange(50) <= 44 + i], 0.1, 0, f"query {i}")
    assert np.isnan(out[3:]).all()


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("qs,ks,vs", [(1, 1, 1e-30), (1, 1, 1e30), (1e-20, 1e20, 1), (1e15, 1e-15, 1e-6), (40, 1, 1), (1e-30, 1, 1)])
def test_scales_far_from_one(fmt, qs, ks, vs):
    c = Cache([300, 1], 1, 128, 16, fmt, seed=5, kscale=ks, vscale=vs)
    q = (qs * torch.randn(2, 8, 128, device="cuda")).to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.09, **c.kw)
    for b, L in enumerate(c.lens):
        check_attention(c, _bf(q)[b], _bf(plan.out)[b], _np(plan.lse)[b].astype(np.float64), [np.ones(L, bool)], 0.09,
                        b, f"length {L}")


def test_value_scales_that_differ_between_tokens():
    # a heavily weighted token with tiny values beside lightly weighted ones with huge values, in both orders
    c = Cache([64, 64], 1, 128, 16, INT4, seed=6)
    for b in range(2):
        for n in range(64):
            big = n % 2 == b
            k = c.K[b][:, n:n + 1] * 0 + (0.0 if big else 1.0)
            v = np.random.default_rng(n).standard_normal((1, 1, 128)) * (1e4 if big else 1e-3)
            row = ref.pack(k.astype(np.float32), v.astype(np.float32))
            c.pool[c.table[b, n // 16], :, n % 16] = torch.from_numpy(row[:, 0]).cuda()
            K, V, ks, vs = ref.unpack(row)
            c.K[b][:, n], c.V[b][:, n], c.ks[b][:, n], c.vs[b][:, n] = K[:, 0], V[:, 0], ks[:, 0], vs[:, 0]
    q = torch.full((2, 8, 128), 1.0, device="cuda").to(torch.bfloat16)
    for scale in (0.05, 0.15, 0.4):
        plan = spa.paged_attend(q=q, sm_scale=scale, **c.kw)
        for b in range(2):
            check_attention(c, _bf(q)[b], _bf(plan.out)[b], _np(plan.lse)[b].astype(np.float64), [np.ones(64, bool)],
                            scale, b, f"scale {scale}")


def test_value_scales_that_differ_within_a_token():
    c = Cache([100], 1, 128, 16, INT4, seed=14)
    rng = np.random.default_rng(14)
    for n in range(100):
        k = rng.standard_normal((1, 1, 128)).astype(np.float32)
        v = rng.standard_normal((1, 1, 128)) * np.repeat(2.0 ** rng.integers(-12, 13, 4), 32)
        v[0, 0, :32] *= n % 7 != 3           # and groups that are zero
        row = ref.pack(k, v.astype(np.float32))
        c.pool[c.table[0, n // 16], :, n % 16] = torch.from_numpy(row[:, 0]).cuda()
        K, V, ks, vs = ref.unpack(row)
        c.K[0][:, n], c.V[0][:, n], c.ks[0][:, n], c.vs[0][:, n] = K[:, 0], V[:, 0], ks[:, 0], vs[:, 0]
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, **c.kw)
    check_attention(c, _bf(q)[0], _bf(plan.out)[0], _np(plan.lse)[0].astype(np.float64), [np.ones(100, bool)], 0.1, 0,
                    "groups")


@pytest.mark.parametrize("fmt,d", [(INT4, 128), (INT4, 64), (BF16, 128)])
def test_a_value_that_is_not_finite_reaches_its_channels_and_no_others(fmt, d):
    c = Cache([70, 70], 1, d, 16, fmt, seed=15)
    host = c.pool.view(torch.uint8).reshape(c.pool.shape[0], 1, 16, -1)
    for b in range(2):                      # one group (4-bit) or one channel (bf16) of one token's value, and of all
        for n in ([33] if b == 0 else range(70)):
            at = slice(d + 8 + 4, d + 8 + 6) if fmt == INT4 else slice(2 * d + 80, 2 * d + 82)
            host[c.table[b, n // 16], 0, n % 16, at] = torch.tensor([0xC0, 0x7F], dtype=torch.uint8, device="cuda")
    q = torch.randn(2, 4, d, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, **c.kw)
    out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
    hit = np.zeros(d, bool)
    hit[slice(d // 2, 3 * d // 4) if fmt == INT4 else slice(40, 41)] = True
    assert np.isnan(out[:, :, hit]).all() and np.isfinite(out[:, :, ~hit]).all() and np.isfinite(lse).all()
    c.V[0][:, :, hit] = c.V[1][:, :, hit] = 0
    out[:, :, hit] = 0
    for b in range(2):
        check_attention(c, _bf(q)[b], out[b], lse[b], [np.ones(70, bool)], 0.1, b, "other channels")


def test_attend_reports_bad_pages_and_skips_them():
    for fmt in (INT4, BF16):
        c = Cache([80], 1, 128, 16, fmt, seed=7)
        c.kw["page_table"][0, 2] = -1
        q = torch.randn(1, 4, 128, device="cuda").to(torch.bfloat16)
        plan = spa.paged_attend(q=q, sm_scale=0.1, **c.kw)
        assert spa.read_device_status(plan.ws) == INVALID
        n = np.arange(80)
        check_attention(c, _bf(q)[0], _bf(plan.out)[0], _np(plan.lse)[0].astype(np.float64), [(n < 32) | (n >= 48)],
                        0.1, 0, "page 2 missing")
        c.kw["kv_len"].fill_(1 << 30)        # clamped to what the table can hold, and reported
        c.kw["page_table"][0, 2] = int(c.table[0, 2])
        plan.run()
        assert spa.read_device_status(plan.ws) == INVALID
        check_attention(c, _bf(q)[0], _bf(plan.out)[0], _np(plan.lse)[0].astype(np.float64), [np.ones(80, bool)],
                        0.1, 0, "length clamped")


def test_many_sequences_and_supports_pass_one_launch():
    # more sequences, and more supports, than one launch takes
    B = 2500
    lens = [(7 * b) % 40 for b in range(B)]
    c = Cache(lens, 1, 64, 16, INT4, seed=8)
    q = torch.randn(B, 2, 64, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.2, **c.kw)
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    for b in list(range(0, B, 97)) + [2047, 2048, 2049, B - 1]:
        check_attention(c, qv[b], out[b], lse[b], [np.ones(lens[b], bool)], 0.2, b, f"sequence {b}")
    idx = np.tile(np.arange(8, dtype=np.int32), (2 * B, 1))
    count = np.minimum(np.repeat(lens, 2), 8)
    plan = spa.paged_attend(q=q, sm_scale=0.2, idx=_i32(idx), count=_i32(count), collapse=spa.SPA_COLLAPSE_NONE, **c.kw)
    out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
    for b in list(range(0, B, 97)) + [1023, 1024, 1025, B - 1]:
        check_attention(c, qv[b], out[b], lse[b], [np.arange(lens[b]) < 8] * 2, 0.2, b, f"supports of {b}")


def test_chunks_of_many_sequences_pass_one_launch():
    B, n = 600, 18                           # 36 rows of each sequence and kv head; some have none of them
    lens = [n + (7 * b) % 150 for b in range(B)]
    news = [n if b % 5 else 0 for b in range(B)]
    news[256] = news[255] = news[512] = 29
    lens[256] = 29
    lens[255] = lens[512] = 160
    start = np.concatenate(([0], np.cumsum(news)))
    c = Cache(lens, 1, 64, 16, INT4, seed=51)
    T = int(start[-1]) + 300 * n             # (rows behind the last sequence count towards the choice of a kernel)
    q = torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.2, seq_start=_i32(start), run=False, **c.kw)
    plan.out.fill_(9)
    plan.run()
    assert spa.read_device_status(plan.ws) == 0
    out, lse, qv = _bf(plan.out), _np(plan.lse).astype(np.float64), _bf(q)
    assert (out[start[-1]:] == 9).all()
    for b in list(range(1, B, 61)) + [255, 256, 257, 511, 512, 513, B - 1]:
        for i in range(news[b]):
            t = start[b] + i
            check_attention(c, qv[t], out[t], lse[t], [np.arange(lens[b]) <= lens[b] - news[b] + i], 0.2, b,
                            f"sequence {b}, query {i}")


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [60, 45]])
def test_scales_of_the_softmax_that_are_not_positive(fmt, new):
    lens = [90, 700]
    c = Cache(lens, 2, 128, 16, fmt, seed=52)
    start = np.concatenate(([0], np.cumsum(new)))
    q = torch.randn(int(start[-1]), 8, 128, device="cuda").to(torch.bfloat16)
    for scale in (-0.1, 0.0):
        plan = spa.paged_attend(q=q, sm_scale=scale, seq_start=_i32(start), **c.kw)
        assert spa.read_device_status(plan.ws) == 0
        out, lse = _bf(plan.out), _np(plan.lse).astype(np.float64)
        for b, (n, L) in enumerate(zip(new, lens)):
            for i in sorted({0, n // 2, n - 1}):
                t = start[b] + i
                # softmax(-s q K) is softmax(s (-q) K)
                check_attention(c, -_bf(q)[t], out[t], lse[t], [np.arange(L) <= L - n + i] * 2, -scale, b,
                                f"scale {scale}, sequence {b}, query {i}")


# ------------------------------------------------------------------------------------------------ as used
def test_decode_loop_in_a_graph_matches_the_oracle():
    """Prompt, then decode steps replayed from one graph: append with rotation, then attention; kv_len on the
    device is the only thing that moves."""
    B, Hkv, G, d, page = 3, 2, 4, 128, 16
    prompt, steps = [5, 40, 17], 40
    c = Cache([0] * B, Hkv, d, page, INT4, fill=False, extra=(max(prompt) + steps) // page + 1)
    rng = np.random.default_rng(9)
    inv = (10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
    invd = torch.from_numpy(inv).cuda()

    def tokens(T):
        return torch.from_numpy(rng.standard_normal((T, (G + 2) * Hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda()

    kv_len, kw = c.kw["kv_len"], c.kw
    kv_len.copy_(_i32(prompt))
    pre = tokens(sum(prompt))
    start = _i32(np.concatenate(([0], np.cumsum(prompt))))
    spa.paged_append(k=pre[:, G * Hkv:(G + 1) * Hkv], v=pre[:, (G + 1) * Hkv:], seq_start=start, inv_freq=invd, **kw)
    new = tokens(B)
    app = spa.paged_append(k=new[:, G * Hkv:(G + 1) * Hkv], v=new[:, (G + 1) * Hkv:], q=new[:, :G * Hkv],
                           inv_freq=invd, run=False, **kw)
    att = spa.paged_attend(q=app.q_out, sm_scale=d**-0.5, run=False, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv_len.add_(1)
        app.run()
        att.run()
    for step in range(steps):
        new.copy_(tokens(B))
        graph.replay()
        if step in (0, 11, steps - 1):
            host = _np(c.pool)
            for b in range(B):
                L = prompt[b] + step + 1
                assert int(kv_len[b]) == L
                rows = np.stack([c.row(host, b, n) for n in range(L)], 1)
                K, V, ks, vs = ref.unpack(rows)
                c.K, c.V, c.ks, c.vs = [K] * B, [V] * B, [ks] * B, [vs] * B
                # the newest row is the rotated new key
                wk = ref.rotate(_bf(new[b:b + 1, G * Hkv:(G + 1) * Hkv]), [L - 1], inv, False)[0]
                assert (np.abs(K[:, -1] - wk) <= np.repeat(ks[:, -1], d // 4, -1) * 0.501 + 1e-5).all()
                wq = ref.rotate(_bf(new[b:b + 1, :G * Hkv]), [L - 1], inv, False)[0]
                assert (np.abs(_bf(app.q_out)[b] - wq) <= 2.0**-8 * np.abs(wq) + 1e-5).all()
                check_attention(c, _bf(app.q_out)[b], _bf(att.out)[b], _np(att.lse)[b].astype(np.float64),
                                [np.ones(L, bool)] * Hkv, d**-0.5, b, f"step {step}, sequence {b}")
    assert spa.read_device_status(app.ws) == 0 and spa.read_device_status(att.ws) == 0


def test_sparse_decode_over_a_paged_cache():
    """append -> low-rank index scores -> top-p selection -> attention on the supports: the supports are those of
    the dense path, and the attention equals sparse_attend on the gathered dense rows up to both roundings."""
    B, Hkv, G, d, page, N = 2, 2, 8, 128, 64, 3000
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(B * N, (G + 2) * Hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    c = Cache([N] * B, Hkv, d, page, INT4, fill=False)
    inv = torch.tensor((10000.0 ** (-np.arange(32) / 32)).astype(np.float32), device="cuda")
    app = spa.paged_append(k=qkv[:, G * Hkv:(G + 1) * Hkv], v=qkv[:, (G + 1) * Hkv:], q=qkv[:, :G * Hkv],
                           seq_start=_i32([0, N, 2 * N]), inv_freq=inv, **c.kw)
    q = app.q_out.reshape(B, N, G * Hkv, d)[:, -1].contiguous()
    q_idx = torch.randn(B, G * Hkv, 16, generator=g, device="cuda").to(torch.bfloat16)
    kidx = torch.randn(B, Hkv, N, 16, generator=g, device="cuda").to(torch.bfloat16)
    scores = spa.index_scores(spa.SPA_SCORE_LOWRANK, q_idx, kidx, None, Hkv, spa.SPA_COLLAPSE_GROUP_MEAN, 1.0)
    idx, count, _ = spa.select_topp(scores, 0.6, 4, 64)
    att = spa.paged_attend(q=q, sm_scale=d**-0.5, idx=idx, count=count, **c.kw)
    dense = spa.paged_gather(N=N, **c.kw)
    want, want32, want_lse = spa.sparse_attend(q, dense.K, dense.V, idx, count, spa.SPA_COLLAPSE_GROUP_MEAN, d**-0.5)
    assert 64 < int(count.min()) and int(count.max()) < N
    # the dense rows round each value to bf16 (2^-8 relative): logits move by at most 2^-8 sum|qk|, outputs by 2^-8 |v|
    rows = np.stack([np.stack([c.row(_np(c.pool), b, n) for n in range(N)], 1) for b in range(B)])
    K, V, ks, vs = ref.unpack(rows)
    c.K, c.V, c.ks, c.vs = list(K), list(V), list(ks), list(vs)
    for b in range(B):
        sees = []
        for h in range(Hkv):
            s = np.zeros(N, bool)
            s[_np(idx)[b * Hkv + h, :int(count[b * Hkv + h])]] = True
            sees.append(s)
        check_attention(c, _bf(q)[b], _bf(att.out)[b], _np(att.lse)[b].astype(np.float64), sees, d**-0.5, b, f"seq {b}")
    assert (att.lse - want_lse).abs().max() <= 0.05 and (att.out.float() - want32).abs().max() <= 0.05


def test_two_plans_on_two_streams_do_not_disturb_each_other():
    cs = [Cache([9000, 31], 2, 128, 16, INT4, seed=s) for s in (11, 12)]
    qs = [torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16) for _ in cs]
    plans = [spa.paged_attend(q=q, sm_scale=0.1, run=False, **c.kw) for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip(plans, streams):
            p.run(s)
    torch.cuda.synchronize()
    for c, q, p in zip(cs, qs, plans):
        assert spa.read_device_status(p.ws) == 0
        for b, L in enumerate(c.lens):
            check_attention(c, _bf(q)[b], _bf(p.out)[b], _np(p.lse)[b].astype(np.float64), [np.ones(L, bool)] * 2, 0.1,
                            b, f"length {L}")


def test_chunks_on_two_streams_and_in_a_graph():
    cs = [Cache([700, 90, 300], 2, d, 16, INT4, seed=s, extra=2) for s, d in ((41, 128), (42, 64))]
    start = [0, 60, 61, 161]
    qs = [torch.randn(161, 8, c.d, device="cuda").to(torch.bfloat16) for c in cs]
    plans = [spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32(start), run=False, **c.kw) for c, q in zip(cs, qs)]
    plans.append(spa.paged_attend(q=qs[0][:3].contiguous(), sm_scale=0.1, run=False, **cs[0].kw))   # and a decode beside them
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip(plans, streams):
            p.run(s)
    torch.cuda.synchronize()

    def check(lens):
        for c, q, p in zip(cs, qs, plans):
            assert spa.read_device_status(p.ws) == 0
            for b in range(3):
                n = start[b + 1] - start[b]
                for i in (0, n - 1):
                    t = start[b] + i
                    check_attention(c, _bf(q)[t], _bf(p.out)[t], _np(p.lse)[t].astype(np.float64),
                                    [np.arange(len(c.K[b][0])) <= lens[b] - n + i] * 2, 0.1, b, f"row {t}")

    check([700, 90, 300])
    check_attention(cs[0], _bf(qs[0])[1], _bf(plans[2].out)[1], _np(plans[2].lse)[1].astype(np.float64),
                    [np.ones(90, bool)] * 2, 0.1, 1, "decode")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plans[0].run()
        plans[1].run()
    for c in cs:                             # shorter sequences, as if tokens had been taken back
        c.kw["kv_len"].copy_(_i32([650, 61, 111]))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check([650, 61, 111])


def test_starts_out_of_order_are_reported():
    # overlapping, negative and too large starts: nothing outside the tensors is touched, the status says so
    for n, fmt in ((3, INT4), (3, BF16), (200, INT4)):
        c = Cache([300] * 4, 1, 64, 16, fmt, seed=43)
        q = torch.randn(n, 4, 64, device="cuda").to(torch.bfloat16)
        for start in ([0, n, 0, n, 1], [5, 4, 3, 2, 1], [-7, 2, 1 << 30, 2, n], [0, 0, 0, 0, n + 9]):
            plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32(start), **c.kw)
            assert spa.read_device_status(plan.ws) == INVALID
            add = spa.paged_append(k=q[:, :1], v=q[:, 1:2], q=q, seq_start=_i32(start), **c.kw)
            assert spa.read_device_status(add.ws) in (0, INVALID)
        good = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32([0, 1, 1, 2, n]), **c.kw)
        assert spa.read_device_status(good.ws) == 0


def test_a_plan_built_on_one_stream_runs_on_another_at_once():
    c = Cache([500], 1, 128, 16, INT4, seed=13)
    s = torch.cuda.Stream()
    q = torch.randn(1, 4, 128, device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    plan = spa.paged_attend(q=q, sm_scale=0.1, run=False, **c.kw)
    with torch.cuda.stream(s):
        plan.run()
    s.synchronize()
    check_attention(c, _bf(q)[0], _bf(plan.out)[0], _np(plan.lse)[0].astype(np.float64), [np.ones(500, bool)], 0.1, 0,
                    "other stream")


def test_python_refusals():
    c = Cache([20, 20], 2, 64, 16, INT4, fill=False)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k=k.float()), dict(v=k[:1]), dict(k=k.cpu()), dict(k=k[:, :, :32]), dict(q_out=q),
                dict(q=q, q_out=q[:1]), dict(inv_freq=torch.zeros(64, device="cuda")),
                dict(positions=_i32([1])), dict(seq_start=_i32([0, 2])), dict(kv_len=c.kw["kv_len"].long())):
        with pytest.raises((TypeError, ValueError)):
            spa.paged_append(**{**dict(k=k, v=k), **c.kw, **bad})
    with pytest.raises(spa.SpaError):       # q_out over q
        spa.paged_append(k=k, v=k, q=q, q_out=q, **c.kw)
    for bad in (dict(q=q[:1]), dict(idx=_i32([[0]])), dict(idx=_i32([[0]]), count=_i32([1])),
                dict(q=torch.cat([q, q]), seq_start=_i32([0, 1, 4]), idx=_i32(np.zeros((4, 1))), count=_i32(np.zeros(4)))):
        with pytest.raises((TypeError, ValueError)):
            spa.paged_attend(**{**dict(q=q, sm_scale=0.1), **c.kw, **bad})
    with pytest.raises(spa.SpaError):       # 17 query heads per kv head
        spa.paged_attend(q=torch.zeros(2, 34, 64, dtype=torch.bfloat16, device="cuda"), sm_scale=0.1, **c.kw)
    with pytest.raises((TypeError, ValueError)):
        spa.paged_gather(N=4, K=k, **c.kw)


def _far(B):
    # two sequences with rows, 0-1 and 3-4, among empty ones, and a start out of order between them
    s = np.full(B + 1, 3, np.int64)
    s[:11], s[11], s[12], s[B] = 0, 2, -4, 5
    return s.tolist()


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("T,start", [(8, [0, 5, 3, 8]), (8, [-2, 3, 8]), (8, [0, 4, 12]), (8, [6, 2, 8, 1]),
                                     (8, [-7, 2, 1 << 30, 2, 8]), (8, [0, 3, 3, -1, 4, 8]), (6, _far(40)), (6, _far(300)),
                                     (6, _far(1500))])
def test_append_reports_starts_out_of_order_and_keeps_to_the_other_sequences(fmt, T, start):
    B, d = len(start) - 1, 64
    ok = [0 <= a <= e <= T for a, e in zip(start, start[1:])]
    lens = [e - a if g else 1 for a, e, g in zip(start, start[1:], ok)]
    c = Cache(lens, 1, d, 16, fmt, fill=False)
    c.pool.view(torch.uint8).fill_(0xA5)
    kv = torch.randn(2, T, 1, d, device="cuda").to(torch.bfloat16)
    q = torch.randn(T, 2, d, device="cuda").to(torch.bfloat16)
    q_out = torch.full_like(q, 7)
    add = spa.paged_append(k=kv[0], v=kv[1], q=q, q_out=q_out, seq_start=_i32(start), **c.kw)
    assert spa.read_device_status(add.ws) == INVALID
    host = _np(c.pool.view(torch.uint8)).reshape(c.pool.shape[0], 1, 16, -1)
    want = np.full_like(host, 0xA5)
    k, v = _bf(kv[0]).astype(np.float32), _bf(kv[1]).astype(np.float32)
    shared = False
    for t in range(T):
        mine = [b for b in range(B) if ok[b] and start[b] <= t < start[b + 1]]
        shared |= len(mine) > 1
        assert torch.equal(q_out[t], q[t] if mine else torch.full_like(q[t], 7))
        if mine:
            n = t - start[mine[0]]
            row = ref.pack(k[t], v[t]) if fmt == INT4 else np.concatenate(
                (ref.bf16_bits(k[t]), ref.bf16_bits(v[t])), -1).astype("<u2").view(np.uint8)
            want[c.table[mine[0], n // 16], :, n % 16] = row
    assert (host == want).all()
    if shared:
        return
    att = spa.paged_attend(q=q, sm_scale=0.2, seq_start=_i32(start), run=False, **c.kw)
    att.out.fill_(9)
    att.run()
    assert spa.read_device_status(att.ws) == INVALID
    if fmt == INT4:
        k, v, ks, vs = ref.unpack(ref.pack(k[:, 0], v[:, 0]))
    for b in range(B):
        if ok[b] and lens[b]:
            a, e = start[b], start[b + 1]
            c.K, c.V = {b: k[a:e].reshape(1, e - a, d)}, {b: v[a:e].reshape(1, e - a, d)}
            if fmt == INT4:
                c.ks, c.vs = {b: ks[None, a:e]}, {b: vs[None, a:e]}
            for i in range(e - a):
                check_attention(c, _bf(q)[a + i], _bf(att.out)[a + i], _np(att.lse)[a + i].astype(np.float64),
                                [np.arange(e - a) <= i], 0.2, b, f"sequence {b}, row {a + i}")
    nobody = [t for t in range(T) if not any(ok[b] and start[b] <= t < start[b + 1] for b in range(B))]
    assert (att.out[nobody] == 9).all()


def test_append_of_many_sequences():
    # more sequences than a warp counts through: rows of each, of empty ones, and of nobody
    B, d = 1500, 64
    new = [(3 * b) % 4 for b in range(B)]
    start = np.concatenate(([0], np.cumsum(new))) + 2
    T = int(start[-1]) + 5
    c = Cache([max(n, 1) for n in new], 1, d, 16, INT4, fill=False)
    c.pool.fill_(0xA5)
    kv = torch.randn(2, T, 1, d, device="cuda").to(torch.bfloat16)
    add = spa.paged_append(k=kv[0], v=kv[1], seq_start=_i32(start), **c.kw)
    assert spa.read_device_status(add.ws) == 0
    want = np.full_like(_np(c.pool), 0xA5)
    rows = ref.pack(_bf(kv[0]).astype(np.float32), _bf(kv[1]).astype(np.float32))
    for b in range(B):
        for i in range(new[b]):
            want[c.table[b, 0], :, i] = rows[start[b] + i]
    assert (_np(c.pool) == want).all()


def test_one_workspace_serves_every_attention_call_in_turn():
    # decode, drafted tokens, chunks of both formats and head sizes, supports: one after the other on one workspace, all of
    # them with units that are split over CTAs
    L = 40_000
    plans = []
    for fmt, d, new in [(INT4, 128, 1), (BF16, 64, 60), (INT4, 128, 5), (INT4, 128, 60), (BF16, 128, 1), (INT4, 64, 1)]:
        c = Cache([L], 1, d, 64, fmt, seed=71, fill=False)
        c.pool.random_(0, 255) if fmt == INT4 else c.pool.normal_()
        if fmt == INT4:                     # any codes will do; scales of one
            c.pool.view(torch.bfloat16)[..., d // 2:] = 1.0
        q = torch.randn(new, 4, d, device="cuda").to(torch.bfloat16)
        plans.append(dict(q=q, sm_scale=0.02, seq_start=_i32([0, new]), **c.kw))
        if new == 1:
            plans.append(dict(q=q, sm_scale=0.02, idx=torch.arange(0, L, 2, dtype=torch.int32, device="cuda")[None],
                              count=_i32([L // 2]), **c.kw))
    alone = [spa.paged_attend(**kw) for kw in plans]
    ws = spa.workspace(max(p.ws.numel() for p in alone))
    shared = [spa.paged_attend(ws=ws, run=False, **kw) for kw in plans]
    for order in (range(len(plans)), reversed(range(len(plans))), [0, 3, 0, 4, 6, 1, 1, 2, 5]):
        for i in order:
            shared[i].out.fill_(9)
            shared[i].run()
            assert torch.equal(shared[i].out, alone[i].out) and torch.equal(shared[i].lse, alone[i].lse), i
    assert spa.read_device_status(ws) == 0


def test_supports_without_room_for_an_entry():
    c = Cache([20, 0], 2, 64, 16, INT4, seed=72)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    for count in (0, 3):                    # (a count above cap is cut)
        plan = spa.paged_attend(q=q, sm_scale=0.1, idx=torch.empty((4, 0), dtype=torch.int32, device="cuda"),
                                count=_i32([count] * 4), run=False, **c.kw)
        plan.out.fill_(9)
        plan.run()
        assert spa.read_device_status(plan.ws) == 0
        assert (plan.out == 0).all() and (plan.lse == -np.inf).all()


@pytest.mark.parametrize("fmt", [INT4, BF16])
@pytest.mark.parametrize("new", [1, 5, 60])
def test_a_pool_without_pages(fmt, new):
    pool = spa.paged_cache(0, 1, 16, 128, fmt)
    kw = dict(cache=pool, page_table=_i32([[0] * 9, [0] * 9]), kv_len=_i32([130, 0]))
    q = torch.randn(new, 4, 128, device="cuda").to(torch.bfloat16)
    plan = spa.paged_attend(q=q, sm_scale=0.1, seq_start=_i32([0, new, new]), run=False, **kw)
    plan.out.fill_(9)
    plan.run()
    assert spa.read_device_status(plan.ws) == INVALID
    assert (plan.out == 0).all() and (plan.lse == -np.inf).all()
    add = spa.paged_append(k=q[:, :1], v=q[:, 1:2], seq_start=_i32([0, new, new]), **kw)
    assert spa.read_device_status(add.ws) == INVALID
    got = spa.paged_gather(N=40, **kw)
    assert spa.read_device_status(got.ws) == INVALID and (got.K == 0).all()


@pytest.mark.parametrize("fmt", [INT4, BF16])
def test_two_tokens_of_one_slot_leave_a_mixture_of_theirs(fmt):
    # sequences that share a page, against the rules: nothing else is written, and every piece is of one of the two
    d = 128
    c = Cache([3, 3], 2, d, 16, fmt, fill=False)
    c.kw["page_table"][1] = c.kw["page_table"][0]
    c.pool.view(torch.uint8).fill_(0xA5)
    kv = torch.randn(2, 2, 2, d, device="cuda").to(torch.bfloat16)
    add = spa.paged_append(k=kv[0], v=kv[1], **c.kw)
    assert spa.read_device_status(add.ws) == 0
    host = _np(c.pool.view(torch.uint8)).reshape(c.pool.shape[0], 2, 16, -1)
    k, v = _bf(kv[0]).astype(np.float32), _bf(kv[1]).astype(np.float32)
    rows = ref.pack(k, v) if fmt == INT4 else np.concatenate((ref.bf16_bits(k), ref.bf16_bits(v)), -1).astype("<u2").view(np.uint8)
    got = host[c.table[0, 0], :, 2].copy().view("<u2")
    a, b = rows[0].copy().view("<u2"), rows[1].copy().view("<u2")
    assert ((got == a) | (got == b)).all()
    host[c.table[0, 0], :, 2] = 0xA5
    assert (host == 0xA5).all()
