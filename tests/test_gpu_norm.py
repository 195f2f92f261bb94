"""GPU RMS norm against the float64 oracle: bf16 output, residual stream, and codes.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
  h        one fp32 sum, one rounding to bf16: u + 2^-8 relative.
  y        sum of squares: at most 64 fused adds per thread and 12 across threads (any K here is below
           64 * 256 elements), so (64 + 12 + 2) u, halved by the square root, + 4 u for the mean, the
           root and the reciprocal, + 2 u for two products + u for h: below DELTA = 48 u.
  codes    quotient within DELTA + 3 u (scale, division): the code must lie between the codes of
           u64 (1 - 2 DELTA) and u64 (1 + 2 DELTA), i.e. equal unless a rounding border is that near.
           The dynamic scale itself is within DELTA + u."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, codes, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DELTA = 48 * U
EPS = 1e-6

# rows x columns: one element, one wave's rows, a workgroup's, several chunks, not a multiple of 8,
# many rows (a wave per row) with 1, 2, 4 and 8 chunks per lane and with the last chunks empty,
# rows long enough for 1024 threads, and longer than any register form
SHAPES = [(1, 1), (3, 7), (1, 64), (5, 200), (2, 2048), (7, 2056), (33, 4096), (3, 11008), (2, 16384), (2, 20000),
          (1, 65544), (1024, 512), (1025, 520), (1027, 1032), (1026, 2048), (1030, 4096), (1024, 4104), (2, 5001)]


def _inputs(seed, M, K):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-6, 7, size=(M, 1))
    r = 3.0 * rng.standard_normal((M, K))
    w = 1.0 + 0.3 * rng.standard_normal(K)
    if M > 2:
        x[1] = 0.0                                     # an all-zero row (with no residual)
        x[-1] *= 1e-12                                 # a row where eps dominates
    b = [oracle.f32_to_bf16_bits(a.astype(np.float32)) for a in (x, r, w)]
    return b, [bits_to_f64(a) for a in b]


def _within(got, ref, rel, what):
    err = np.abs(got - ref)
    worst = np.max(err - rel * np.abs(ref))
    assert worst <= 1e-30, f"{what}: {worst:.3e} beyond {rel:.3e} relative"


def _check_codes(got, y64, s, qtype, what):
    """got: raw codes; y64 / s within 2 DELTA of the quotient that was coded."""
    u = y64 / s
    lo, hi = np.minimum(u * (1 - 2 * DELTA), u * (1 + 2 * DELTA)), np.maximum(u * (1 - 2 * DELTA), u * (1 + 2 * DELTA))
    if qtype == "int8":
        g = got.view(np.int8).astype(np.float64)
        lo, hi = np.clip(np.rint(lo), -127, 127), np.clip(np.rint(hi), -127, 127)
    else:
        g = oracle.e4m3fn_decode(got).astype(np.float64)
        lo = oracle.e4m3fn_decode(oracle.e4m3fn_encode_sat(lo.astype(np.float32)))
        hi = oracle.e4m3fn_decode(oracle.e4m3fn_encode_sat(hi.astype(np.float32)))
    bad = (g < lo) | (g > hi)
    assert not bad.any(), f"{what}: {bad.sum()} codes off, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("MK", SHAPES)
def test_norm_matches_the_oracle(MK, residual):
    M, K = MK
    print(f"norm M={M} K={K} residual={residual}", flush=True)
    (xb, rb, wb), (x, r, w) = _inputs(M * 7 + K, M, K)
    y64, h64 = layer.rms_norm(x, w, EPS, r if residual else None)
    xg, rg, wg = bf16_to_gpu(xb), bf16_to_gpu(rb) if residual else None, bf16_to_gpu(wb)
    rel_y = 2.0 ** -8 + 2 * DELTA

    def h_of(got, n):
        if not residual:
            return got if isinstance(got, tuple) else (got,)
        _within(bits_to_f64(bf16_bits(got[n])), h64, 2.0 ** -8 + 2 * U, "h")
        return got

    y = h_of(qlq.rms_norm(xg, wg, EPS, residual=rg), 1)[0]
    _within(bits_to_f64(bf16_bits(y)), y64, rel_y, "y")
    for qtype, qmax in (("int8", 127.0), ("fp8_e4m3fn", 448.0)):
        got = h_of(qlq.rms_norm_quant_dynamic(xg, wg, qtype, EPS, residual=rg), 2)
        s = got[1].cpu().numpy().astype(np.float64)
        am = np.abs(y64).max(axis=1)
        s64 = np.where(am == 0, 1.0, am / qmax)
        assert np.all(np.abs(s - s64) <= (DELTA + 2 * U) * s64), "scale"
        _check_codes(codes(got[0]), y64, s[:, None], qtype, f"dynamic {qtype}")
        s_in = np.float32(3.1 / qmax)                  # saturates some values
        got = h_of(qlq.rms_norm_quant_static(xg, wg, float(s_in), qtype, EPS, residual=rg), 1)
        _check_codes(codes(got[0]), y64, np.float64(s_in), qtype, f"static {qtype}")


def test_codes_are_the_quotients_roundings():
    # without a residual h is x itself; h w, its product with a factor that fp64 gives, and (dynamic) the largest
    # |h w| are rounded once each, so a code can differ from the float64 quotient's only within 3 u of a border
    near = 3 * U * (1 + 2.0 ** -10)
    for (M, K), qtype in (((1200, 2048), "int8"), ((1100, 1536), "fp8_e4m3fn"), ((40, 5001), "int8"), ((9, 12000), "fp8_e4m3fn")):
        rng = np.random.default_rng(K)
        xb, wb = (oracle.f32_to_bf16_bits(a.astype(np.float32)) for a in (rng.standard_normal((M, K)), 1 + 0.3 * rng.standard_normal(K)))
        y64, _ = layer.rms_norm(bits_to_f64(xb), bits_to_f64(wb), EPS)
        qmax = 127.0 if qtype == "int8" else 448.0
        s = np.float32(np.abs(y64).max() / qmax)
        x, w = bf16_to_gpu(xb), bf16_to_gpu(wb)
        static = codes(qlq.rms_norm_quant_static(x, w, float(s), qtype, EPS))
        dynamic = codes(qlq.rms_norm_quant_dynamic(x, w, qtype, EPS)[0])
        for got, quotient in ((static, y64 / np.float64(s)), (dynamic, y64 / (np.abs(y64).max(1, keepdims=True) / qmax))):
            if qtype == "int8":
                g = got.view(np.int8).astype(np.float64)
                border = np.abs(quotient - g) - 0.5 - near * np.abs(quotient)    # beyond the half step
            else:
                g = oracle.e4m3fn_decode(got).astype(np.float64)
                step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(quotient), 2.0 ** -20))) - 3, -9)
                border = np.abs(quotient - g) / step - 0.5 - near * np.abs(quotient) / step
            over = (border > 2.0 ** -40) & (np.abs(quotient) <= qmax)
            assert not over.any(), f"{M}x{K} {qtype}: {over.sum()} codes on the other side of a border"


@pytest.mark.parametrize("MK", [(5, 2048), (1024, 1000), (3, 77), (2, 70000)])
def test_norm_in_place_equals_out_of_place(MK):
    M, K = MK
    (xb, rb, wb), _ = _inputs(11, M, K)
    wg = bf16_to_gpu(wb)
    y, h = qlq.rms_norm(bf16_to_gpu(xb), wg, EPS, residual=bf16_to_gpu(rb))
    for y_is_x in (True, False):
        x, r = bf16_to_gpu(xb), bf16_to_gpu(rb)
        qlq.rms_norm(x, wg, EPS, residual=r, out=x if y_is_x else r, residual_out=r if y_is_x else x)
        a, b = (x, r) if y_is_x else (r, x)
        assert torch.equal(a, y) and torch.equal(b, h)
    r = bf16_to_gpu(rb)
    c, s, h2 = qlq.rms_norm_quant_dynamic(bf16_to_gpu(xb), wg, "int8", EPS, residual=r, residual_out=r)
    c0, s0, _ = qlq.rms_norm_quant_dynamic(bf16_to_gpu(xb), wg, "int8", EPS, residual=bf16_to_gpu(rb))
    assert h2.data_ptr() == r.data_ptr() and torch.equal(r, h)
    assert torch.equal(c, c0) and torch.equal(s, s0)


@pytest.mark.parametrize("shift", [1, 4])
def test_norm_at_odd_addresses(shift):
    # element-aligned views of a larger buffer: not 16-byte aligned
    M, K = 6, 1024
    (xb, rb, wb), (x, r, w) = _inputs(5, M, K)
    buf = torch.zeros(M * K + shift, dtype=torch.bfloat16, device=dev())
    xg = buf[shift:].view(M, K)
    xg.copy_(bf16_to_gpu(xb))
    y, h = qlq.rms_norm(xg, bf16_to_gpu(wb), EPS, residual=bf16_to_gpu(rb))
    y64, h64 = layer.rms_norm(x, w, EPS, r)
    _within(bits_to_f64(bf16_bits(y)), y64, 2.0 ** -8 + 2 * DELTA, "y")
    _within(bits_to_f64(bf16_bits(h)), h64, 2.0 ** -8 + 2 * U, "h")
    out = torch.full((M * K + 8,), 77, dtype=torch.int8, device=dev())
    c, s = qlq.rms_norm_quant_dynamic(xg, bf16_to_gpu(wb), "int8", EPS, out=out[shift:shift + M * K].view(M, K))
    c2, s2 = qlq.rms_norm_quant_dynamic(bf16_to_gpu(xb), bf16_to_gpu(wb), "int8", EPS)
    y64, _ = layer.rms_norm(x, w, EPS)
    _check_codes(codes(c), y64, s.cpu().numpy().astype(np.float64)[:, None], "int8", "odd address")
    assert bool((out[:shift] == 77).all()) and bool((out[shift + M * K:] == 77).all())


def test_norm_extreme_static_scales():
    # scales whose reciprocal leaves the range of the product form take the IEEE division
    (xb, _, wb), (x, _, w) = _inputs(9, 4, 256)
    y64, _ = layer.rms_norm(x, w, EPS)
    for s_in in (1e-38, 1e-9, 3e38):
        c = qlq.rms_norm_quant_static(bf16_to_gpu(xb), bf16_to_gpu(wb), s_in, "int8", EPS)
        _check_codes(codes(c), y64, np.float64(np.float32(s_in)), "int8", f"scale {s_in}")


def test_norm_binding_refusals_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev())
    w = torch.ones(64, dtype=torch.bfloat16, device=dev())
    for call in (lambda: qlq.rms_norm(x.t(), w), lambda: qlq.rms_norm(x, w[:32]), lambda: qlq.rms_norm(x.float(), w),
                 lambda: qlq.rms_norm(x, w.float()), lambda: qlq.rms_norm(x, w.cpu()),
                 lambda: qlq.rms_norm(x, w, residual=x[:2]), lambda: qlq.rms_norm(x, w, residual_out=x),
                 lambda: qlq.rms_norm(x, w, out=x.float()),
                 lambda: qlq.rms_norm_quant_dynamic(x, w, "int8", x_scale=torch.zeros(3, device=dev())),
                 lambda: qlq.rms_norm_quant_static(x, w, 1.0, "int8", out=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qlq.QlqError):
        qlq.rms_norm(x, w, eps=0.0)
    with pytest.raises(qlq.QlqError):
        qlq.rms_norm(x, w, residual=x, out=x, residual_out=x)
