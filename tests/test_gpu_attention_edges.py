"""Attention over the 8-bit cache where the softmax or its masks are at their limits.

Weights far below a row's largest: w_t = 2^(x_t - m) goes to fp16 with the largest weight 2^15, so a weight is off
by at most 2^-11 of itself or, below 2^-14, by 2^-25, i.e. by 2^-40 of the largest.  With n tokens, V = max |v| and
S = sum_t p_t |v_t| an output is off by at most 2^-8 of itself (bf16), (2^-11 + 2 E) S and n 2^-40 V, E the
exponent's error: scores are single products here (one channel of q is not zero), so E = u (3 (2 A + 56) + n / 32 + 40)
with u = 2^-24 and A the largest score (test_gpu_attention.py has the terms)."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle.layer import kv_attention, slots_of
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, dev
from tests.test_gpu_attention import Problem

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _gpu(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a)).view(dt).to(dev())


@pytest.mark.parametrize("octaves", [20.0, 25.2, 33.0])
@pytest.mark.parametrize("heads", [(4, 1, 64), (4, 4, 128), (8, 2, 96), (2, 1, 192), (2, 1, 256), (3, 1, 32)])
@pytest.mark.parametrize("BL", [(1, 32), (300, 3000)])
def test_tail_far_below_the_largest_weight(BL, heads, octaves):
    # One token outweighs every other by `octaves`, and half of the channels are zero in its values: there the
    # output is the others' alone.  32 tokens are one wave's; of the long sequences (which share their pages) a
    # wave takes hundreds and more.
    (B, L), (Hq, Hk, D) = BL, heads
    print(f"tail B={B} L={L} heads={heads} octaves={octaves}", flush=True)
    rng = np.random.default_rng(L + D)
    page = 32
    pages = -(-L // page)
    P, top = pages * page, L // 3
    kc = np.zeros((P, Hk, D), np.int8)
    kc[:, :, 1:] = rng.integers(-127, 128, size=(P, Hk, D - 1))
    kc[top, :, 0] = 64
    vc = rng.integers(0x30, 0x7F, size=(P, Hk, D)).astype(np.uint8)          # 0.5 .. 448
    vc[top, :, ::2] = 0
    ks, vs = np.full((P, Hk, D // 32), 2.0 ** -6, np.float16), np.full((P, Hk), 2.0 ** -8, np.float16)
    q = np.zeros((Hq, D), np.float32)
    q[:, 0] = octaves * np.log(2.0) * (1 + np.arange(Hq) / 256)
    qb = oracle.f32_to_bf16_bits(q)
    table = torch.arange(pages, dtype=torch.int32, device=dev()).expand(B, pages).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device=dev())
    cache = qlq.QuantizedKV(_gpu(kc, torch.int8), _gpu(ks, torch.float16), _gpu(vc, torch.uint8), _gpu(vs, torch.float16))
    lse = torch.zeros(B, Hq, device=dev())
    out = qlq.kv_attention(bf16_to_gpu(np.tile(qb, (B, 1, 1))), cache, table, lens, page, scale=1.0, lse=lse)
    k = kc.astype(np.float64) * 2.0 ** -6
    v = oracle.e4m3fn_decode(vc).astype(np.float64) * 2.0 ** -8
    q64 = bits_to_f64(qb)
    got, got_lse = bits_to_f64(bf16_bits(out)), lse.cpu().numpy().astype(np.float64)
    for h in range(Hq):
        s = k[:L, h // (Hq // Hk)] @ q64[h]
        p = np.exp(s - s.max())
        l64 = s.max() + np.log(p.sum())
        p /= p.sum()
        o64 = p @ v[:L, h // (Hq // Hk)]
        E = U * (3 * (2 * np.abs(s).max() + 56) + L / 32 + 40)
        bound = 2.0 ** -8 * o64 + (2.0 ** -11 + 2 * E) * o64 + L * 2.0 ** -40 * np.abs(v).max()      # (v >= 0: S = o)
        over = np.abs(got[:, h] - o64) / bound
        assert over.max() <= 1.0, f"head {h}: {over.max():.2f} times the bound"
        assert np.abs(got_lse[:, h] - l64).max() <= 2 * E + U * abs(l64)


@pytest.mark.parametrize("case", [((1, 1, 1), (40, 20, 90), "few rows"), ((1, 1), (9000, 700), "few rows, joined"),
                                  ((150, 40), (150, 300), "many rows"), ((90,), (3000,), "many rows, joined")])
def test_a_query_with_nan_is_nan_in_its_own_row_alone(case):
    nqs, lens, what = case
    print(f"NaN query: {what}", flush=True)
    for Hq, Hk, D in ((4, 2, 64), (4, 1, 128)):
        p = Problem(sum(lens) + D, nqs, lens, Hq, Hk, D, 16, each=False)
        lse0, lse = torch.zeros(p.T, Hq, device=dev()), torch.zeros(p.T, Hq, device=dev())
        out0 = p.run(lse=lse0).clone()
        hit = [(0, 1), (p.T - 1, 3)]
        for t, h in hit:
            p.q[t, h, 5] = float("nan")
        out = p.run(lse=lse)
        for t, h in hit:
            assert bool(torch.isnan(out[t, h]).all()) and bool(torch.isnan(lse[t, h])), what
            out[t, h], lse[t, h] = out0[t, h], lse0[t, h]
        assert torch.equal(out, out0) and torch.equal(lse, lse0), what


@pytest.mark.parametrize("window", [1, 5, 40, 333])
@pytest.mark.parametrize("nqs", [(1, 1, 1), (3, 1, 9), (150, 64, 80)])
def test_entries_before_the_window_may_hold_anything(nqs, window):
    # what no query can see any more (a page that its owner gave back may be another's, half written) changes nothing
    lens = [n + e for n, e in zip(nqs, (700, 1003, 90))]
    print(f"entries before the window nqs={nqs} window={window}", flush=True)
    for Hq, Hk, D in ((4, 2, 64), (2, 1, 96), (4, 1, 128), (2, 1, 256)):
        p = Problem(sum(nqs) + D + window, nqs, lens, Hq, Hk, D, 16, each=max(nqs) == 1)
        out = p.check(window=window, what="before")
        lse, lse2 = torch.zeros(p.T, Hq, device=dev()), torch.zeros(p.T, Hq, device=dev())
        p.run(window=window, lse=lse)
        for scale in (float("nan"), float("inf")):
            for b, (n, L) in enumerate(zip(nqs, lens)):
                gone = slots_of(p.table[b], max(0, L - n - window + 1), 16, p.pool)
                at = torch.from_numpy(gone).to(dev())
                p.cache.k_codes[at], p.cache.v_codes[at] = 127, 0x7F
                p.cache.k_scales[at], p.cache.v_scales[at] = scale, scale
            same = torch.equal(p.run(window=window, lse=lse2), out) and torch.equal(lse2, lse)
            assert same, (Hq, Hk, D, scale)


MANY = [  # query tokens of each sequence (8 heads of 32 over one KV head: a tile of 256 rows is 32 of them)
    ("one sequence of 67 tiles", (2129,)),
    ("65 tiles and a bit, then more", (2080, 1, 0, 37)),
    ("64 tiles end with a sequence", (1024, 1000, 24, 0, 33, 2)),
    ("sequences across the 64th tile", (40, 1500, 0, 700, 3, 64)),
    ("70 sequences", tuple(9 + b % 5 for b in range(70))),
    ("131 sequences, some empty, one long", tuple(0 if b % 7 == 3 else 12 + b % 3 for b in range(130)) + (900,))]


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("case", MANY, ids=[c[0] for c in MANY])
def test_many_query_tiles_and_sequences(case, window):
    what, nqs = case
    lens = [n + (b * 13) % 50 for b, n in enumerate(nqs)]
    print(f"many tiles: {what}, window {window}", flush=True)
    p = Problem(sum(nqs) + window, nqs, lens, 8, 1, 32, 16, each=False)
    p.check(window=window, what=what)


@pytest.mark.parametrize("nqs", [(1, 1, 1), (90, 40)])
def test_lengths_and_tables_that_the_graph_itself_changes(nqs):
    # a captured step that first advances the lengths and swaps in the next step's block table, both on the device
    lens = [n + e for n, e in zip(nqs, (200, 900, 37))]
    p = Problem(sum(nqs), nqs, [L + 8 for L in lens], 4, 1, 128, 16, each=max(nqs) == 1)
    other = Problem(sum(nqs) + 1, nqs, [L + 8 for L in lens], 4, 1, 128, 16, each=max(nqs) == 1)
    first = torch.tensor(lens, dtype=torch.int32, device=dev())
    pages = p.pool // 16                               # two tables over one pool: the second one's pages behind
    assert other.pool == p.pool and other.bt.shape == p.bt.shape
    c = [torch.cat(t) for t in zip(*((q.cache.k_codes, q.cache.k_scales, q.cache.v_codes, q.cache.v_scales) for q in (p, other)))]
    cache = qlq.QuantizedKV(*c)
    own = (other.bt >= 0) & (other.bt < pages)
    tables = [torch.where((p.bt >= 0) & (p.bt < pages), p.bt, -1), torch.where(own, other.bt + pages, -1)]
    both, step = torch.stack(tables), torch.zeros(1, dtype=torch.int64, device=dev())
    sl, bt = first.clone(), tables[0].clone()
    out, lse = torch.empty_like(p.q), torch.empty(p.T, 4, device=dev())

    def body():
        step.add_(1)
        sl.add_(1)
        bt.copy_(both[step % 2][0])
        qlq.kv_attention(p.q, cache, bt, sl, 16, q_start=p.q0, out=out, lse=lse)

    body()                                             # (set-up outside the capture)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        body()
    step.zero_()
    sl.copy_(first)
    for n in range(1, 9):
        want_lse = torch.empty_like(lse)
        want = qlq.kv_attention(p.q, cache, tables[n % 2], first + n, 16, q_start=p.q0, lse=want_lse)
        out.zero_()
        g.replay()
        same = torch.equal(out, want) and torch.equal(lse, want_lse)
        assert same, n


@pytest.mark.parametrize("heads", [(4, 1, 32), (4, 2, 64), (4, 1, 128), (8, 2, 256)])
@pytest.mark.parametrize("huge", [2.0 ** 14, 2.0 ** 24])
def test_prompt_rows_that_do_not_see_a_huge_value(heads, huge):
    # One token's values are 2^14 or 2^24 times the others'.  Rows before it do not see it, and their bound does not
    # know it: 2^-8 of the output and (2 2^-11 + 2 E) S as for any prompt (test_gpu_attention.py), and what fp16's
    # smallest step (2^-24) leaves of a value at the outlier's scaling (its own scale at 2^5 or more, a code at 2^-8):
    # half a step is 2^-30 of the outlier's scale, once per token.
    Hq, Hk, D = heads
    nqs, lens = (100, 70), (260, 70)
    p = Problem(D, nqs, lens, Hq, Hk, D, 16, each=False)
    kc, ks, vc, vs = p.host
    at = [slots_of(p.table[b], lens[b], 16, p.pool) for b in range(2)]
    for b, s in enumerate(at):                         # queries 0 .. 59 of each sequence come before it
        t = lens[b] - nqs[b] + 60
        vs[s[t]] = oracle.fp16_encode(np.minimum(oracle.fp16_decode(vs[s[t]]) * huge, 65504.0).astype(np.float32))
    p.cache = qlq.QuantizedKV(_gpu(kc, torch.int8), _gpu(ks.view(np.int16), torch.float16), _gpu(vc, torch.uint8),
                              _gpu(vs.view(np.int16), torch.float16))
    got = bits_to_f64(bf16_bits(p.run()))
    k, v = p.values()
    q = bits_to_f64(p.qb)
    o64, _, _, S = kv_attention(q, k, v, p.table, lens, 16, p.starts)
    for b, s in enumerate(at):
        ku, scales = np.abs(k[s]), oracle.fp16_decode(vs[s]).astype(np.float64)
        A = D ** -0.5 * max((np.abs(q[:, h]) @ ku[:, h // (Hq // Hk)].T).max() for h in range(Hq))
        A1 = D ** -0.5 * np.abs(q).max() * ku.sum(-1).max()
        E = U * (42 * A + A1 + 3 * (2 * A + 56) + lens[b] / 32 + 40) + 2.0 ** -11 * A + U * A1
        rows = slice(p.starts[b], p.starts[b] + 60)
        unseen = lens[b] - nqs[b] + 60
        V = np.abs(v[s[:unseen]]).max()
        bound = 2.0 ** -8 * np.abs(o64[rows]) + S[rows] * (2 * 2.0 ** -11 + 2 * E) + lens[b] * 2.0 ** -32 * V
        bound += 2.0 ** -30 * scales.max()
        over = np.abs(got[rows] - o64[rows]) / bound
        assert over.max() <= 1.0, f"sequence {b}: {over.max():.2f} times the bound"


@pytest.mark.parametrize("heads", [(4, 1, 32), (4, 2, 64), (4, 1, 128), (8, 2, 256)])
def test_prompt_rows_that_do_not_see_a_huge_key(heads):
    # One token's keys have scales of 3000; the others' are small (2^-6).  A query is the key of its own token, scaled
    # to a score of 8.  Rows before the huge one do not see it; in their bound A and A' are those of the keys they see,
    # and a key beside the huge one is off by fp16's smallest half step at 2^-7 of it: 2^-18, times scale sum |q| in a
    # score.
    Hq, Hk, D = heads
    nqs, lens = (100, 70), (260, 70)
    p = Problem(D + 1, nqs, lens, Hq, Hk, D, 16, each=False)
    kc, ks, vc, vs = p.host
    at = [slots_of(p.table[b], lens[b], 16, p.pool) for b in range(2)]
    for s in at:
        ks[s] = oracle.fp16_encode((oracle.fp16_decode(ks[s]) * 2.0 ** -6).astype(np.float32))
    k, v = p.values()
    q = np.concatenate([np.repeat(k[s[lens[b] - nqs[b]:]], Hq // Hk, axis=1) for b, s in enumerate(at)])
    q *= 8 * D ** 0.5 / (q * q).sum(-1, keepdims=True)
    p.qb = oracle.f32_to_bf16_bits(q.astype(np.float32))
    p.q = bf16_to_gpu(p.qb)
    for b, s in enumerate(at):                         # queries 0 .. 59 of each sequence come before it
        ks[s[lens[b] - nqs[b] + 60]] = oracle.fp16_encode(np.float32(3000.0))
    p.cache = qlq.QuantizedKV(_gpu(kc, torch.int8), _gpu(ks.view(np.int16), torch.float16), _gpu(vc, torch.uint8),
                              _gpu(vs.view(np.int16), torch.float16))
    lse = torch.zeros(p.T, Hq, device=dev())
    got = bits_to_f64(bf16_bits(p.run(lse=lse)))
    q, (k, v) = bits_to_f64(p.qb), p.values()
    o64, l64, _, S = kv_attention(q, k, v, p.table, lens, 16, p.starts)
    for b, s in enumerate(at):
        unseen = lens[b] - nqs[b] + 60
        ku, vu, rows = np.abs(k[s[:unseen]]), np.abs(v[s[:unseen]]), slice(p.starts[b], p.starts[b] + 60)
        qa = np.abs(q[rows])
        A = D ** -0.5 * max((qa[:, h] @ ku[:, h // (Hq // Hk)].T).max() for h in range(Hq))
        A1 = D ** -0.5 * qa.max() * ku.sum(-1).max()
        E = U * (42 * A + A1 + 3 * (2 * A + 56) + lens[b] / 32 + 40) + 2.0 ** -11 * A + U * A1
        E += 2.0 ** -18 * D ** -0.5 * qa.sum(-1).max()
        off = np.abs(lse.cpu().numpy()[rows] - l64[rows]) / (2 * E + U * np.abs(l64[rows]))
        bound = 2.0 ** -8 * np.abs(o64[rows]) + S[rows] * (2 * 2.0 ** -11 + 2 * E) + lens[b] * 2.0 ** -32 * vu.max()
        over = np.abs(got[rows] - o64[rows]) / bound
        assert max(over.max(), off.max()) <= 1.0, f"sequence {b}: output {over.max():.2f}, lse {off.max():.2f} times the bound"
