"""8-bit integer operands: codes and scales against the nearest integers of exact quotients, and the
product bit for bit (its sums are exact, so the outputs are float32 operations rounded once)."""

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from oracle import int8
from parity_util import DEV, to_dev

pytestmark = pytest.mark.gpu
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
TYPES = pytest.mark.parametrize("dtype", ["bf16", "f16"])


# -------------------------------------------------------------------------------------- quantize

def bits_of(x, dtype):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(TORCH[dtype]).view(torch.int16).numpy().view(np.uint16)


def check_quantize(bits, dtype):
    x = to_dev(bits, dtype)
    rows, cols = bits.shape
    full = torch.full((rows * cols + 256,), 85, dtype=torch.int8, device=DEV)
    scales = torch.full((rows + 64,), -5.0, device=DEV)
    q = full[:rows * cols].view(rows, cols)
    fp8.int8_quantize_rowwise(x, q=q, scales=scales[:rows])
    torch.cuda.synchronize()
    want, s = int8.quantize_rowwise(bits, dtype)
    assert (full[rows * cols:] == 85).all() and (scales[rows:] == -5.0).all()
    assert np.array_equal(np.nan_to_num(scales[:rows].cpu().numpy(), nan=-3.0), np.nan_to_num(s, nan=-3.0))
    got = q.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    again = fp8.int8_quantize_rowwise(x)
    assert torch.equal(again[0], q)


@TYPES
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 16), (2, 511), (2, 512), (300, 520), (7, 1000), (300, 1024), (3, 2048), (300, 2050),
                                       (2, 4096), (300, 4096), (2, 5000), (260, 8192), (3, 14336), (260, 10000), (2, 16384), (2, 16400), (3, 20001)])
def test_quantize_sizes(rows, cols, dtype):
    rng = np.random.default_rng(rows * cols)
    check_quantize(bits_of(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 3), dtype), dtype)


@TYPES
def test_quantize_every_value_under_many_scales(dtype):
    """All 2^16 patterns of the type in rows whose largest magnitude is each of many: among them ties, and scales so small
    that remainders leave float32's normal numbers."""
    every = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    inf = 0x7F80 if dtype == "bf16" else 0x7C00
    rng = np.random.default_rng(1)
    tops = np.unique(np.concatenate([[1, 2, 3, 100, 127, 254, inf - 1], rng.integers(1, inf, 60), inf - 128 * np.arange(1, 5)]))
    if dtype == "bf16":
        tops = np.concatenate([tops, 127 + 128 * np.arange(0, 255, 16)])          # largest significands of many exponents
    rows = []
    for top in tops:
        x = every[(every & 0x7FFF) <= top]
        rows.append(np.concatenate([x, np.zeros(65536 - len(x), np.uint16)]))
    check_quantize(np.stack(rows), dtype)


@TYPES
def test_quantize_ties(dtype):
    """Rows whose scale is a power of two, so that x / s falls on halves exactly."""
    x = np.concatenate([np.arange(-254, 255) / 2, [127.0] * 3])
    check_quantize(bits_of(np.stack([x * 2.0 ** e for e in (0, -3, 5, -10)]), dtype), dtype)


@TYPES
@pytest.mark.parametrize("cols", [16, 700, 5000, 17000, 33])
def test_quantize_specials(cols, dtype):
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((6, cols))
    x[0] = 0
    x[1, cols // 2] = np.nan
    x[2, 3], x[2, 4] = np.inf, np.nan
    x[3, cols - 1] = -np.inf
    x[4] = -0.0
    check_quantize(bits_of(x, dtype), dtype)


def test_quantize_empty():
    for shape in ((0, 16), (5, 0)):
        q, s = fp8.int8_quantize_rowwise(torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        assert q.shape == shape and s.tolist() == [1.0] * shape[0]


# --------------------------------------------------------------------------------------- product

def operands(M, N, K, seed=0, low=-128):
    g = torch.Generator().manual_seed(seed)
    qa, qb = (torch.randint(low, 128, (r, K), generator=g, dtype=torch.int8) for r in (M, N))
    sa, sb = (torch.rand(r, generator=g) * 0.02 + 1e-3 for r in (M, N))
    return qa, sa, qb, sb


def check_gemm(ops, dtype, where="random"):
    M, N = ops[0].shape[0], ops[2].shape[0]
    full = torch.full((M * N + 512,), -7.0, dtype=TORCH[dtype], device=DEV)
    out = full[:M * N].view(M, N)
    dev = [t.to(DEV) for t in ops]
    got = fp8.int8_gemm_scaled_rowwise(*dev, out=out)
    torch.cuda.synchronize()
    assert got is out and (full[M * N:] == -7.0).all()
    _, want = int8.gemm_rowwise(*(t.numpy() for t in ops))
    want = torch.from_numpy(want).to(TORCH[dtype])
    bad = (out.cpu() != want).nonzero()
    assert len(bad) == 0, (where, len(bad), bad[:4].tolist())
    assert torch.equal(fp8.int8_gemm_scaled_rowwise(*dev, out_dtype=TORCH[dtype]), out)


@TYPES
@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 17, 32, 33, 64, 65, 128, 129, 200])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 144), (130, 128), (515, 1024), (1000, 2064), (96, 4096)])
def test_products(M, N, K, dtype):
    check_gemm(operands(M, N, K, seed=M), dtype)


@pytest.mark.parametrize("M,N,K", [(300, 5632, 256), (1024, 1100, 512), (600, 9000, 128), (4100, 4200, 128), (2048, 9000, 256), (257, 640, 2000)])
def test_large_tiles(M, N, K):
    check_gemm(operands(M, N, K, seed=N), "bf16")


@pytest.mark.parametrize("M,N,K", [(300, 5632, 272), (1024, 1100, 528), (600, 9000, 144), (4100, 4200, 112), (2048, 9000, 240), (300, 300, 16),
                                   (129, 5, 1568), (2255, 1961, 352), (4096, 4400, 6160), (21, 700, 9264), (128, 130, 1008), (33, 46, 13392)])
def test_last_slab_of_every_length(M, N, K):
    """K % 128 != 0: zeros of A stand against whatever lies behind a row of B."""
    ops = operands(M, N, K, seed=K)
    check_gemm(ops, "f16" if K % 32 else "bf16")


@TYPES
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 13, 16, 17])
@pytest.mark.parametrize("M,K", [(17, 144), (130, 2064), (1000, 1024), (4099, 16), (20000, 112)])
def test_few_channels_of_many_tokens(M, N, K, dtype):
    check_gemm(operands(M, N, K, seed=N), dtype)


@pytest.mark.parametrize("M,N", [(0, 5), (5, 0), (0, 0)])
def test_empty_products(M, N):
    out = fp8.int8_gemm_scaled_rowwise(*(t.to(DEV) for t in operands(M, N, 32)))
    assert out.shape == (M, N) and out.dtype == torch.bfloat16


@pytest.mark.parametrize("M", [1, 3, 9, 40, 130])
def test_largest_sums(M):
    """K at its limit with codes of -128 and 127 only: sums up to 2^31 - 2^18, exact."""
    K, N = 131056, 24
    qa, sa, qb, sb = operands(M, N, K, seed=M)
    qa[:], qb[:] = -128, -128
    qb[1::2] = 127
    qa[M // 2:, ::3] = 127
    if M > 1:
        assert int(qa[0].long() @ qb[0].long()) == 128 * 128 * K
    check_gemm((qa, sa, qb, sb), "bf16")


@TYPES
@pytest.mark.parametrize("M", [1, 3, 20, 150])
def test_scales_that_are_not_finite(M, dtype):
    """A row's or a column's scale reaches its own outputs only; outputs past the type are infinite."""
    qa, sa, qb, sb = operands(M, 70, 256, seed=3)
    qa[0, 0] += qa[0, 0] == 0
    good = fp8.int8_gemm_scaled_rowwise(*(t.to(DEV) for t in (qa, sa, qb, sb)), out_dtype=TORCH[dtype])
    sa2, sb2 = sa.clone(), sb.clone()
    sa2[M - 1], sb2[5], sb2[6] = float("nan"), float("inf"), 3e38
    out = fp8.int8_gemm_scaled_rowwise(*(t.to(DEV) for t in (qa, sa2, qb, sb2)), out_dtype=TORCH[dtype])
    keep = [c for c in range(70) if c not in (5, 6)]
    assert torch.equal(out[:M - 1][:, keep], good[:M - 1][:, keep]) and out[M - 1].isnan().all()
    _, want = int8.gemm_rowwise(qa.numpy(), sa2.numpy(), qb.numpy(), sb2.numpy())
    want = torch.from_numpy(want).to(TORCH[dtype])
    assert torch.equal(out.cpu().nan_to_num(3.0), want.nan_to_num(3.0))


def test_quantized_layer():
    """Activations quantized on the way into weights quantized once, against float64: each code is off by half a step at
    most, so an output by sum (|a| sb + |b| sa + sa sb / 2) / 2 and the roundings."""
    g = torch.Generator(device=DEV).manual_seed(7)
    x, w = (torch.empty(s, device=DEV).normal_(generator=g).bfloat16() for s in ((37, 512), (130, 512)))
    (qa, sa), (qb, sb) = fp8.int8_quantize_rowwise(x), fp8.int8_quantize_rowwise(w)
    out = fp8.int8_gemm_scaled_rowwise(qa, sa, qb, sb).double()
    a, b, sa, sb = x.double(), w.double(), sa.double()[:, None], sb.double()[None]
    want = a @ b.T
    bound = (a.abs().sum(1, keepdim=True) * sb + b.abs().sum(1)[None] * sa + 512 * sa * sb / 2) / 2 * (1 + 2 ** -20)
    assert ((out - want).abs() <= bound + 2.0 ** -8 * out.abs() * 1.01).all()
    assert float((out - want).norm() / want.norm()) < 0.02


def test_binding_refuses_on_the_gpu():
    qa, sa, qb, sb = (t.to(DEV) for t in operands(4, 8, 32))
    for error, args in ((ValueError, (qa, sa[:3], qb, sb)), (ValueError, (qa, sa, qb[:, :16].contiguous(), sb)), (TypeError, (qa, sa.double(), qb, sb)),
                        (ValueError, (qa, sa, qb, sb.cpu()))):
        with pytest.raises(error):
            fp8.int8_gemm_scaled_rowwise(*args)
    with pytest.raises(fp8.Fp8Error, match="BAD_SHAPE"):
        fp8.int8_gemm_scaled_rowwise(qa[:, :24].contiguous(), sa, qb[:, :24].contiguous(), sb)
    with pytest.raises(ValueError, match="overlaps"):
        fp8.int8_gemm_scaled_rowwise(qa, sa, qb, sb, out=qb.view(torch.bfloat16).view(-1)[:32].view(4, 8))


def test_stream_and_graph():
    """Quantize and product on a side stream, and in a graph replayed with eager work between."""
    x = torch.randn(64, 1024, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    _, _, qb, sb = (t.to(DEV) for t in operands(1, 300, 1024, seed=2))

    def layer(q=None, s=None, out=None):
        q, s = fp8.int8_quantize_rowwise(x, q=q, scales=s)
        return fp8.int8_gemm_scaled_rowwise(q, s, qb, sb, out=out)

    want = layer().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
    side.synchronize()
    assert torch.equal(got, want)
    q, s, out = torch.empty((64, 1024), dtype=torch.int8, device=DEV), torch.empty(64, device=DEV), torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(q, s, out)
    for _ in range(3):
        out.zero_()
        q.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        _ = (want.float() * 2).sum()
