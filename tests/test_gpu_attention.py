"""GPU attention over the paged 8-bit cache against the float64 oracle.

Tolerance, from the arithmetic (u = 2^-24, one fp32 rounding), for an output channel with
S = sum_t p_t |v_t|, n tokens seen, A = max_t scale sum_c |q_c k_c| and V = max |v|:
  scores    fp32 sums of products exact in fp32: 32 products per channel group in the matrix unit and the
            groups after one another, (40 + 2) u A; q in fp16 after its power-of-two scaling: 2^-11 2^-14
            of the row's largest channel, below u A' with A' = max|q| sum|k| scale <= 64 A for the inputs
            here (bounded below by measuring A'); the exponent's own roundings 3 u (|x| + 16), |x| <= 2 A + 40
  weights   rounded to fp16: 2^-11 relative, or 2^-25 of the largest weight below fp16's normal range:
            n 2^-25 V in the output; exp2, log2, reciprocal: 8 u
  sums      (n / 32 + 32) u
so |out - out64| <= 2^-8 |out64| + S (2^-11 + 2 E) + n 2^-25 V, E = u (42 A + A' + 3 (2 A + 56) + n / 32 + 40),
and |lse - lse64| <= 2 E + u |lse|.
Many query rows (per KV head and sequence, on average, more than 32 for heads of 96 and 128, 64 for others): K and V are rounded to 11 bits after their
scales as well, 2^-11 of a product, so E grows by 2^-11 A (and by 2^-25 scale sum|q| below fp16's normal range,
less than A' u for the keys here) and the output's error by 2^-11 S."""
import math

import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Problem:
    """A cache whose pages hold the sequences' tokens and poison (NaN codes and scales) everywhere else."""

    def __init__(self, seed, nqs, lens, Hq, Hk, D, page, spare=2, each=True, qgain=1.0):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hk, self.D, self.page, self.lens, self.nqs = Hq, Hk, D, page, list(lens), list(nqs)
        B = len(lens)
        need = [-(-L // page) for L in lens]
        pages = sum(need) + spare
        width = max(max(need), 1) + 1
        order = rng.permutation(pages)
        table = np.full((B, width), 1 << 30, np.int64)              # entries of no token: never read
        table[rng.random((B, width)) < 0.5] = -7
        at = 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.table, self.pool = table, pages * page
        P = self.pool
        kc = np.full((P, Hk, D), 127, np.int8)
        ks = np.full((P, Hk, D // 32), 0x7E00, np.uint16)           # NaN
        vc = np.full((P, Hk, D), 0x7F, np.uint8)                    # NaN
        vs = np.full((P, Hk), 0x7C00, np.uint16)                    # inf
        for b in range(B):
            s = layer.slots_of(table[b], lens[b], page, P)
            if lens[b] == 0:
                continue
            gain = 2.0 ** rng.integers(-3, 4, size=(lens[b], Hk, 1))
            k = rng.standard_normal((lens[b], Hk, D)) * (1 + 4 * (rng.random((1, Hk, D)) < 0.05))
            v = rng.standard_normal((lens[b], Hk, D)) * gain
            e = oracle.kv_quantize(*(oracle.f32_to_bf16_bits(a.astype(np.float32)) for a in (k, v)))
            for dst, src in zip((kc, ks, vc, vs), e):
                dst[s] = src
        self.host = (kc, ks, vc, vs)
        to = lambda a, dt: torch.from_numpy(a).view(dt).to(dev())
        self.cache = qlq.QuantizedKV(to(kc, torch.int8), to(ks.view(np.int16), torch.float16), to(vc, torch.uint8),
                                     to(vs.view(np.int16), torch.float16))
        T = sum(nqs)
        self.T = T
        self.qb = oracle.f32_to_bf16_bits((qgain * rng.standard_normal((T, Hq, D))).astype(np.float32))
        self.q = bf16_to_gpu(self.qb)
        self.bt = torch.from_numpy(table.astype(np.int32)).to(dev())
        self.sl = torch.tensor(lens, dtype=torch.int32, device=dev())
        starts = np.concatenate([[0], np.cumsum(nqs)])
        self.starts = starts
        self.q0 = None if each and all(n == 1 for n in nqs) else torch.from_numpy(starts.astype(np.int32)).to(dev())

    def values(self):
        kc, ks, vc, vs = self.host
        P, Hk, D = kc.shape
        with np.errstate(invalid="ignore"):
            k = (kc.reshape(P, Hk, D // 32, 32) * oracle.fp16_decode(ks)[..., None]).reshape(P, Hk, D)
            v = oracle.e4m3fn_decode(vc).astype(np.float64) * oracle.fp16_decode(vs)[..., None]
        return k, v

    def run(self, **kw):
        return qlq.kv_attention(self.q, self.cache, self.bt, self.sl, self.page, q_start=self.q0, **kw)

    def check(self, scale=None, causal=True, window=0, what=""):
        lse = torch.full((self.T, self.Hq), 123.0, device=dev())
        out = self.run(scale=scale, causal=causal, window=window, lse=lse)
        k, v = self.values()
        self.compare(out, lse, k, v, self.table, self.lens, scale, causal, window, what)
        return out

    def compare(self, out, lse, k, v, table, lens, scale=None, causal=True, window=0, what=""):
        q = bits_to_f64(self.qb)
        sc = self.D ** -0.5 if scale is None else scale
        o64, l64, written, S = layer.kv_attention(q, k, v, table, lens, self.page, self.starts, sc, causal, window)
        used = np.concatenate([layer.slots_of(table[b], lens[b], self.page, self.pool) for b in range(len(lens))]
                              + [np.array([], np.int64)]).astype(np.int64)
        used = used[used >= 0]
        ku, vu = np.abs(k[used]), np.abs(v[used])
        n = max(lens)
        V = vu.max() if used.size else 0.0
        # bounds of A and A' over every pair
        A1 = abs(sc) * np.abs(q).max() * ku.sum(-1).max() if used.size else 0.0
        A = A1 if used.size == 0 else abs(sc) * max(
            (np.abs(q[:, h]) @ ku[:, h // (self.Hq // self.Hk)].T).max() for h in range(self.Hq))
        E = U * (42 * A + A1 + 3 * (2 * A + 56) + n / 32 + 40)
        wide = -(-self.T // len(lens)) * (self.Hq // self.Hk) > (32 if self.D in (96, 128) else 64)
        W = 2.0 ** -11
        if wide:
            E, W = E + 2.0 ** -11 * A + U * A1, 2 * W
        got = bits_to_f64(bf16_bits(out))
        assert np.all(np.isfinite(got)), what
        over = np.abs(got - o64) - (2.0 ** -8 * np.abs(o64) + S * (W + 2 * E) + n * 2.0 ** -25 * V + 1e-38)
        assert np.max(over) <= 0, f"{what}: {np.max(over):.3e} beyond the bound at {np.unravel_index(over.argmax(), over.shape)}"
        if lse is not None:
            lg = lse.cpu().numpy().astype(np.float64)
            empty = np.isneginf(l64)
            assert np.array_equal(np.isneginf(lg), empty), what
            if (~empty).any():
                d = np.abs(lg[~empty] - l64[~empty]) - (2 * E + U * np.abs(l64[~empty]))
                assert d.max() <= 0, f"{what}: lse {d.max():.3e} beyond the bound"


LENS = [0, 1, 31, 32, 33, 63, 100, 255, 256, 257, 1000, 2049]


@pytest.mark.parametrize("heads", [(1, 1, 32), (4, 4, 64), (28, 4, 128), (3, 1, 96), (16, 2, 192), (8, 2, 256),
                                   (20, 1, 128), (40, 1, 64)])
@pytest.mark.parametrize("page", [16, 256])
def test_single_tokens_ragged_lengths(heads, page):
    Hq, Hk, D = heads
    print(f"attention heads={heads} page={page}", flush=True)
    p = Problem(Hq + D + page, [1] * len(LENS), LENS, Hq, Hk, D, page)
    a = p.check(what="decode")
    p.q0 = torch.from_numpy(p.starts.astype(np.int32)).to(dev())     # the same through q_start
    b = p.check(what="decode through q_start")
    assert a.shape == b.shape


@pytest.mark.parametrize("page", [16, 32, 64, 128, 4096])
def test_page_sizes(page):
    p = Problem(page, [1, 1, 1], [5, 33, 300], 4, 2, 64, page)
    p.check(what=f"page {page}")


@pytest.mark.parametrize("window", [0, 1, 7, 64, 100000])
@pytest.mark.parametrize("nqs", [(1, 2, 5, 33), (17, 0, 1, 64), (130, 3, 0, 0), (4, 40, 300, 9)])
def test_many_query_tokens(nqs, window):
    lens = [max(n, 1) + e for n, e in zip(nqs, (300, 0, 31, 1000))]
    print(f"attention nqs={nqs} lens={lens} window={window}", flush=True)
    for Hq, Hk, D in ((4, 2, 64), (7, 1, 128)):
        p = Problem(sum(nqs) + window, nqs, lens, Hq, Hk, D, 16, each=False)
        p.check(window=window, what=f"{Hq},{Hk},{D}")


@pytest.mark.parametrize("heads", [(2, 2, 32), (6, 2, 96), (4, 1, 192), (3, 1, 256)])
def test_many_query_tokens_head_dims(heads):
    Hq, Hk, D = heads
    p = Problem(D, (50, 3, 20), (90, 200, 20), Hq, Hk, D, 64, each=False)
    p.check(what=f"{heads}")


def test_no_causal_mask_scale_and_large_scores():
    p = Problem(5, (9, 1), (77, 130), 4, 2, 64, 32, each=False)
    p.check(causal=False, what="no mask")
    p.check(scale=0.0, what="scale 0: a plain mean")
    p.check(scale=-0.3, what="negative scale")
    p = Problem(6, (1, 1), (900, 40), 4, 2, 64, 32, qgain=2.0 ** 6)   # softmax of one token nearly everywhere
    p.check(what="large scores")
    p = Problem(7, (1, 1), (900, 40), 4, 2, 64, 32, qgain=2.0 ** -40)
    p.check(what="tiny queries")


def test_more_queries_than_tokens_leave_rows_empty():
    p = Problem(8, (5, 40, 3), (2, 0, 3), 4, 2, 64, 16, each=False)
    out = p.check(what="nq > L")
    assert not out[:3].any() and not out[5:45].any()


def test_rows_outside_the_sequences_and_lengths_out_of_range():
    # q rows before the first and behind the last sequence stay as they were; q_start and seq_lens that
    # leave their ranges are bounded (T rows, max_pages * page_size tokens), and pages outside the pool are left out
    p = Problem(9, (2, 1, 3), (40, 20, 80), 4, 2, 64, 16, each=False)
    T = p.T + 4
    q = torch.zeros((T, 4, 64), dtype=torch.bfloat16, device=dev())
    q[2:2 + p.T] = p.q
    out = torch.full_like(q, 3.0)
    lse = torch.full((T, 4), 3.0, device=dev())
    q0 = (p.q0 + 2).contiguous()
    qlq.kv_attention(q, p.cache, p.bt, p.sl, 16, q_start=q0, out=out, lse=lse)
    k, v = p.values()
    p.compare(out[2:2 + p.T].contiguous(), lse[2:2 + p.T], k, v, p.table, p.lens)
    assert bool((out[:2] == 3.0).all()) and bool((out[2 + p.T:] == 3.0).all())
    assert bool((lse[:2] == 3.0).all()) and bool((lse[2 + p.T:] == 3.0).all())
    # a negative length is empty; a length above the table's tokens stops there
    sl = torch.tensor([-5, 20, 1 << 30], dtype=torch.int32, device=dev())
    out2 = qlq.kv_attention(q, p.cache, p.bt, sl, 16, q_start=q0)
    cap = p.table.shape[1] * 16
    p.compare(out2[2:2 + p.T].contiguous(), None, k, v, p.table, [0, 20, cap], what="bounded lengths")
    # q_start beyond T: bounded, nothing written outside
    wild = torch.tensor([2, 4, 5, 1 << 30], dtype=torch.int32, device=dev())
    guard = torch.full((T + 64, 4, 64), 3.0, dtype=torch.bfloat16, device=dev())
    qlq.kv_attention(q, p.cache, p.bt, p.sl, 16, q_start=wild, out=guard[:T])
    assert bool((guard[T:] == 3.0).all()) and bool((guard[:2] == 3.0).all())


def test_bad_pages_are_left_out():
    p = Problem(10, (1, 1, 4), (100, 64, 90), 4, 2, 64, 16, each=False)
    t = p.table.copy()
    t[0, 2], t[1, :], t[2, 0], t[2, 5] = -1, p.pool // 16, 1 << 30, -(1 << 31)
    out = torch.zeros((p.T, 4, 64), dtype=torch.bfloat16, device=dev())
    lse = torch.zeros((p.T, 4), device=dev())
    qlq.kv_attention(p.q, p.cache, torch.from_numpy(t.astype(np.int32)).to(dev()), p.sl, 16, q_start=p.q0, out=out,
                     lse=lse)
    k, v = p.values()
    p.compare(out, lse, k, v, t, p.lens, what="bad pages")
    assert not out[1].any()


def test_strided_queries_and_shared_pages():
    # q as a view of a projection's output; two sequences that share pages (a common prefix)
    p = Problem(11, (1, 1, 1), (200, 150, 90), 8, 2, 128, 16)
    wide = torch.zeros((3, 12 * 128), dtype=torch.bfloat16, device=dev())
    q = wide.as_strided((3, 8, 128), (12 * 128, 128, 1), 0)
    q.copy_(p.q)
    assert torch.equal(qlq.kv_attention(q, p.cache, p.bt, p.sl, 16), p.run())
    t = p.table.copy()
    t[1, :5] = t[0, :5]
    out = qlq.kv_attention(p.q, p.cache, torch.from_numpy(t.astype(np.int32)).to(dev()), p.sl, 16)
    k, v = p.values()
    p.compare(out, None, k, v, t, p.lens, what="shared pages")


def test_long_context_is_split_and_repeats_bit_for_bit():
    p = Problem(12, (1,), (40001,), 7, 1, 64, 256)
    a = p.check(what="one long sequence")
    for _ in range(3):
        assert torch.equal(p.run(), a)
    ws = torch.zeros(qlq.kv_attention_workspace_bytes(1, 1, 7, 1, 64), dtype=torch.uint8, device=dev())
    assert ws.numel() > 0
    for _ in range(3):
        assert torch.equal(p.run(workspace=ws), a)
        assert not ws[:262144].any(), "arrival counters left at zero"
    # one workspace for calls of different shapes on one stream
    p2 = Problem(13, (1,) * 5, (3000, 10, 500, 1, 2500), 4, 4, 128, 64)
    big = torch.zeros(max(ws.numel(), qlq.kv_attention_workspace_bytes(5, 5, 4, 4, 128)), dtype=torch.uint8, device=dev())
    b = p2.check(what="five")
    for _ in range(2):
        assert torch.equal(p.run(workspace=big), a) and torch.equal(p2.run(workspace=big), b)


def test_mixed_batch_of_prefill_and_decode():
    p = Problem(14, (1, 200, 1, 1, 7), (1500, 260, 3, 700, 7), 8, 2, 128, 64, each=False)
    p.check(what="mixed")


@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (5, 1, 96), (3, 1, 32), (2, 1, 256), (6, 3, 192)])
@pytest.mark.parametrize("nqs", [(300, 1, 0, 40), (64, 64), (1000,)])
def test_prompt_chunks(heads, nqs):
    # hundreds of query rows per KV head: whole and partial row tiles, prefixes of none to some, windows
    Hq, Hk, D = heads
    lens = [n + e for n, e in zip(nqs, (0, 700, 5, 333))]
    print(f"prompt chunks heads={heads} nqs={nqs}", flush=True)
    p = Problem(sum(nqs) + D, nqs, lens, Hq, Hk, D, 16 if D % 64 else 64, each=False)
    p.check(what="causal")
    p.check(window=70, what="window")
    if len(nqs) == 2:
        p.check(causal=False, scale=-0.2, what="no mask, negative scale")


def test_prompt_chunk_scales_of_every_size():
    # K scales above 512 and V scales over 25 octaves within one tile and from tile to tile
    p = Problem(22, (100, 70), (300, 260), 4, 2, 64, 32, each=False, qgain=2.0 ** -14)
    kc, ks, vc, vs = p.host
    rng = np.random.default_rng(5)
    for b in range(2):
        s = layer.slots_of(p.table[b], p.lens[b], p.page, p.pool)
        big = s[rng.random(s.size) < 0.02]
        ks[big] = oracle.fp16_encode(np.full(ks[big].shape, 3000.0, np.float32))
        vs[s] = oracle.fp16_encode((2.0 ** rng.uniform(-12, 13, size=vs[s].shape)).astype(np.float32))
    to = lambda a, dt: torch.from_numpy(a).view(dt).to(dev())
    p.cache = qlq.QuantizedKV(to(kc, torch.int8), to(ks.view(np.int16), torch.float16), to(vc, torch.uint8),
                              to(vs.view(np.int16), torch.float16))
    p.check(what="scales of every size")


def test_prompt_chunk_bad_pages_and_empty_rows():
    p = Problem(23, (90, 64, 80), (200, 64, 40), 4, 2, 64, 16, each=False)      # the last: more queries than tokens
    t = p.table.copy()
    t[0, 2], t[1, :], t[0, 7] = -1, p.pool // 16, 1 << 30
    out = torch.full((p.T, 4, 64), 9.0, dtype=torch.bfloat16, device=dev())
    lse = torch.zeros((p.T, 4), device=dev())
    qlq.kv_attention(p.q, p.cache, torch.from_numpy(t.astype(np.int32)).to(dev()), p.sl, 16, q_start=p.q0, out=out,
                     lse=lse)
    k, v = p.values()
    p.compare(out, lse, k, v, t, p.lens, what="bad pages")
    assert not out[90:154].any() and not out[154:194].any()


def test_prompt_chunks_repeat_bit_for_bit_and_share_a_workspace():
    p = Problem(24, (333, 50), (900, 2000), 8, 2, 128, 64, each=False)
    a = p.run()
    p2 = Problem(25, (1,) * 5, (3000, 10, 500, 1, 2500), 4, 4, 128, 64)
    b = p2.run()
    need = max(qlq.kv_attention_workspace_bytes(p.T, 2, 8, 2, 128, one_each=False),
               qlq.kv_attention_workspace_bytes(5, 5, 4, 4, 128))
    ws = torch.zeros(need, dtype=torch.uint8, device=dev())
    for _ in range(3):
        assert torch.equal(p.run(workspace=ws), a) and torch.equal(p2.run(workspace=ws), b)
        assert not ws[:262144].any()


def test_many_sequences():
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 60, size=200)]
    p = Problem(15, (1,) * 200, lens, 2, 1, 64, 16)
    p.check(what="200 sequences")
    nqs = [int(x) for x in rng.integers(0, 4, size=150)]
    p = Problem(16, nqs, [n + int(e) for n, e in zip(nqs, rng.integers(0, 50, size=150))], 2, 1, 64, 16, each=False)
    p.check(what="150 sequences of 0 to 3 queries")


def test_two_streams_at_once():
    p = Problem(17, (1,), (30000,), 4, 1, 64, 256)
    p2 = Problem(18, (1, 1), (20000, 9000), 4, 1, 64, 256)
    a, b = p.run(), p2.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            outs.append((p.run(), a))
        with torch.cuda.stream(s2):
            outs.append((p2.run(), b))
    torch.cuda.synchronize()
    for got, want in outs:
        assert torch.equal(got, want)


def test_captured_and_replayed_with_changing_lengths():
    # two graphs and eager calls on the same stream: each graph has a workspace of its own; the lengths and the
    # block table are read on the device at every replay
    p = Problem(19, (1, 1), (9000, 4000), 4, 1, 64, 256)
    full = p.sl.clone()
    short = torch.tensor([33, 4000], dtype=torch.int32, device=dev())
    out = torch.empty_like(p.q)
    want = p.run().clone()
    p.sl = short
    want_short = p.run().clone()
    p.sl = full.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(out=out)
        graphs.append(g)
    for i in range(6):
        p.sl.copy_(short if i % 3 == 1 else full)
        out.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_short if i % 3 == 1 else want), i
        assert torch.equal(p.run(), want_short if i % 3 == 1 else want), i      # eager between the replays


def test_two_graphs_replayed_at_once():
    # a token's split attention and a prompt chunk's, each captured, replayed on two streams together
    ps = [Problem(30, (1,), (30000,), 4, 1, 64, 256), Problem(31, (150, 40), (1000, 700), 4, 2, 128, 64, each=False)]
    want = [p.run().clone() for p in ps]
    outs, graphs = [torch.empty_like(p.q) for p in ps], []
    for p, o in zip(ps, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for p, o, w in zip(ps, outs, want):
            assert torch.equal(o, w)
            assert torch.equal(p.run(), w)


@pytest.mark.parametrize("heads", [(34, 1, 128), (72, 1, 64), (130, 2, 96), (128, 1, 192), (1024, 1, 32), (1024, 1024, 32),
                                   (331, 331, 32)])
def test_single_tokens_of_many_heads(heads):
    # one query token with more rows than a subtile, or than the many-row kernel's tile; more heads than workgroups
    Hq, Hk, D = heads
    print(f"attention heads={heads}", flush=True)
    p = Problem(Hq + Hk + D, [1] * 4, [0, 1, 65, 200], Hq, Hk, D, 16)
    p.check(what=f"{heads}")


@pytest.mark.parametrize("nqs", [(1, 1), (90, 70)])
def test_offsets_beyond_four_gigabytes(nqs):
    Hk, D, page = 8, 256, 256
    pool = (((1 << 32) // (Hk * D)) // page + 3) * page
    small = Problem(20, nqs, (500, 300), 8, Hk, D, page)
    pages = small.pool // page
    big = qlq.QuantizedKV(torch.empty((pool, Hk, D), dtype=torch.int8, device=dev()),
                          torch.empty((pool, Hk, D // 32), dtype=torch.float16, device=dev()),
                          torch.empty((pool, Hk, D), dtype=torch.uint8, device=dev()),
                          torch.empty((pool, Hk), dtype=torch.float16, device=dev()))
    at = pool - pages * page                           # the sequences' pages at the pool's end
    for a, b in ((big.k_codes, small.cache.k_codes), (big.k_scales, small.cache.k_scales),
                 (big.v_codes, small.cache.v_codes), (big.v_scales, small.cache.v_scales)):
        a[at:] = b
    bt = torch.where((small.bt >= 0) & (small.bt < pages), small.bt + at // page, small.bt)
    out = qlq.kv_attention(small.q, big, bt, small.sl, page, q_start=small.q0)
    assert torch.equal(out, small.run())


def test_unwritten_entries_of_a_fresh_cache():
    # a fresh cache's entries count as zero keys and values; a zero V scale counts as the smallest one
    c = qlq.kv_cache(64, 2, 64)
    c.v_scales.zero_()
    q = bf16_to_gpu(oracle.f32_to_bf16_bits(np.ones((1, 4, 64), np.float32)))
    lse = torch.zeros(1, 4, device=dev())
    out = qlq.kv_attention(q, c, torch.tensor([[0, 1]], dtype=torch.int32, device=dev()),
                           torch.tensor([40], dtype=torch.int32, device=dev()), 32, lse=lse)
    assert not out.any() and torch.allclose(lse, torch.full_like(lse, math.log(40.0)), rtol=1e-6)


def test_attention_binding_refusals_on_the_gpu():
    p = Problem(21, (1, 1), (20, 30), 4, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device=dev())
    bad = [lambda: qlq.kv_attention(p.q.float(), p.cache, p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt.long(), p.sl, 16),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt, p.sl.long(), 16),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt, p.sl[:1], 16),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt, p.sl, 16, q_start=torch.zeros(2, **i32)),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt.cpu(), p.sl, 16),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt, p.sl, 16, out=p.q.float()),
           lambda: qlq.kv_attention(p.q, p.cache, p.bt, p.sl, 16, lse=torch.zeros(2, 3, device=dev())),
           lambda: qlq.kv_attention(p.q, qlq.kv_cache(64, 2, 96), p.bt, p.sl, 16),
           lambda: qlq.kv_attention(p.q.transpose(1, 2), p.cache, p.bt, p.sl, 16)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for kw in (dict(page_size=24), dict(page_size=16, window=-1), dict(page_size=16, scale=math.nan),
               dict(page_size=16, workspace=torch.zeros(256, dtype=torch.uint8, device=dev()))):
        with pytest.raises(qlq.QlqError):
            qlq.kv_attention(p.q, p.cache, p.bt, p.sl, **kw)
