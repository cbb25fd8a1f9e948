"""Input gradient of the frozen projection, dX = dY C^T D^T, for every layer format."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import dictionary_compressed_linear_b200 as dp  # noqa: E402
import synth  # noqa: E402
from oracle import forward as F  # noqa: E402
from oracle.pack import pack_coeff, pack_coeff_blocks, pack_coeff_fmt, pack_dictionary  # noqa: E402

U16 = 2.0 ** -11


def stream():
    return torch.cuda.current_stream().cuda_stream


def projection(d_in, k, d_out, fmt, M, seed=0, rho=0.3):
    """(group, layer) on the device and the oracle's dense D (d_in, k) and C (k, d_out) in fp64."""
    D = synth.gen_dictionary(40, seed, 0, d_in, k)
    gen = synth.gen_coeff_blocks if fmt == "blocks" else synth.gen_coeff
    C = gen(40, seed, 0, 0, k, d_out, rho)
    g = dp.dictproj_pack_group(D, M)
    args = (C.col_ptr, C.atom_idx, C.vals, k, d_out)
    if fmt == "blocks":
        l, pk = dp.dictproj_pack_layer_blocks(*args), pack_coeff_blocks(*args)
        (atoms, vals), ptr = F.decode_coeff_block_entries(pk), pk["blk_ptr"].astype(np.int64) * 16
    elif fmt in ("u8", "bitmap"):
        l = (dp.dictproj_pack_layer if fmt == "u8" else dp.dictproj_pack_layer_bitmap)(*args)
        pk = pack_coeff(*args)
        (atoms, vals), ptr = F.decode_coeff_entries(pk), pk["col_ptr"].astype(np.int64)
    else:
        l, pk = dp.dictproj_pack_layer_fmt(*args, fmt), pack_coeff_fmt(*args, fmt)
        (atoms, vals), ptr = F.decode_coeff_fmt_entries(pk), pk["col_ptr"].astype(np.int64)
    dense = np.zeros((k, d_out))
    np.add.at(dense, (atoms, np.repeat(np.arange(d_out), np.diff(ptr))), vals)
    dp.dictproj_group_reserve_backward(g, d_out)
    cuda = lambda a: torch.tensor(a, device="cuda")  # noqa: E731
    return g, l, cuda(F.decode_dictionary(pack_dictionary(D))), cuda(dense)


def test_few_rows_round_once():
    # up to 32 rows dZ keeps two parts (22 bits): what is left is dX's own rounding, a third of its bound in
    # the mean square, and the fp32 sums
    g, l, D, C = projection(1376, 1040, 1000, "u8", 32)
    dY = torch.randn(32, 1000, generator=torch.Generator().manual_seed(3)).half().cuda()
    dX = torch.empty(32, 1376, dtype=torch.float16, device="cuda")
    dp.dictproj_backward_input(dY.data_ptr(), 32, l, g, dX.data_ptr(), stream())
    torch.cuda.synchronize()
    want = (dY.double() @ C.T) @ D.T
    assert (dX.double() - want).norm().item() <= 1.1 * U16 / math.sqrt(3) * want.norm().item()


def check(dX, dY, D, C):
    """Two roundings to fp16 (dZ and dX) and two fp32 sums. Element by element the worst case: half a step
    of dX, half a step of every dZ (2^-25 at least) carried through |D|, and 2^-23 of the absolute sum for each
    of the d_out + k terms. Over all elements: each rounding's mean square is a third of its bound's square."""
    d_out, k = dY.shape[1], D.shape[1]
    dZ = dY.double() @ C.T
    want = dZ @ D.T
    err = (dX.double() - want).abs()
    sums = (dY.double().abs() @ C.T.abs()) @ D.T.abs()
    bound = U16 * want.abs() + 2.0 ** -25 + (U16 * dZ.abs() + 2.0 ** -25) @ D.T.abs() + 2.0 ** -23 * (d_out + k) * sums
    assert (err <= bound).all(), (err / bound).max().item()
    if want.numel() >= 4096:
        assert err.norm().item() <= 2 * U16 / math.sqrt(3) * want.norm().item()


@pytest.mark.parametrize("M", [1, 32, 33, 129, 300])
def test_every_batch_rounds_once(M):
    # dX is the fp16 value nearest to (exact + delta). delta: a part of dZ is off by at most 2^-16 of its element (two
    # bf16 parts), a third of that squared in the mean square; the fp32 sums are a random walk of 2^-23 a term, with a
    # factor 4 of room. It moves a result to the neighbouring value, a step of at most 2^-10 of it away, with
    # probability |delta| / step, so that the squared difference from the rounded exact result is |delta| step on the
    # average: at most |delta| |step| in norms (Cauchy-Schwarz). A dZ in one fp16 part differs by 3e-4.
    d_in, k, d_out = 1376, 1040, 1000
    g, l, D, C = projection(d_in, k, d_out, "u8", M)
    dY = torch.randn(M, d_out, generator=torch.Generator().manual_seed(3)).half().cuda()
    dX = torch.empty(M, d_in, dtype=torch.float16, device="cuda")
    dp.dictproj_backward_input(dY.data_ptr(), M, l, g, dX.data_ptr(), stream())
    torch.cuda.synchronize()
    want = (dY.double() @ C.T) @ D.T
    delta = 2.0 ** -16 / math.sqrt(3) + 4 * 2.0 ** -23 * math.sqrt(d_out + 2 * k)
    assert (dX.double() - want.half().double()).norm().item() <= math.sqrt(delta * 2.0 ** -10) * want.norm().item()


@pytest.mark.parametrize("M", [5, 100])
@pytest.mark.parametrize("power", [-30, -16, 16, 30])
def test_dz_has_the_range_of_fp32(M, power):
    # a power of two moved from C to D changes dZ's size and nothing else: the same bits
    D, C = synth.gen_dictionary(40, 0, 0, 256, 128), synth.gen_coeff(40, 0, 0, 0, 128, 200, 0.3)
    dY = torch.randn(M, 200, generator=torch.Generator().manual_seed(M)).half().cuda()
    out = []
    for e in (0, power):
        g = dp.dictproj_pack_group((D * np.float32(2.0 ** -e)).astype(np.float32), M)
        l = dp.dictproj_pack_layer(C.col_ptr, C.atom_idx, (C.vals * np.float32(2.0 ** e)).astype(np.float32), 128, 200)
        dp.dictproj_group_reserve_backward(g, 200)
        dX = torch.empty(M, 256, dtype=torch.float16, device="cuda")
        dp.dictproj_backward_input(dY.data_ptr(), M, l, g, dX.data_ptr(), stream())
        torch.cuda.synchronize()
        out.append(dX)
    assert torch.isfinite(out[0]).all() and out[0].abs().max() > 0
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("M", [9, 200])
def test_an_infinity_or_nan_stays_in_its_row(M):
    g, l, D, C = projection(544, 272, 328, "u8", M)
    dY = torch.randn(M, 328, generator=torch.Generator().manual_seed(M)).half().cuda()
    clean, dX = (torch.empty(M, 544, dtype=torch.float16, device="cuda") for _ in range(2))
    dp.dictproj_backward_input(dY.data_ptr(), M, l, g, clean.data_ptr(), stream())
    bad = [1, M // 2, M - 1]
    dY[1, 7], dY[M // 2, 0], dY[M - 1] = float("inf"), float("nan"), -float("inf")
    dp.dictproj_backward_input(dY.data_ptr(), M, l, g, dX.data_ptr(), stream())
    torch.cuda.synchronize()
    keep = [m for m in range(M) if m not in bad]
    assert torch.equal(dX[keep], clean[keep])
    assert not torch.isfinite(dX[bad]).any()


SHAPES = [(32, 16, 8, 1), (256, 128, 200, 5), (544, 272, 328, 37), (1376, 1040, 1000, 129), (4096, 2048, 4096, 64), (288, 304, 72, 300)]


FORMATS = ["u8", "bitmap", "blocks", "fp16", "fp8", "int8"]


@pytest.mark.parametrize("d_in,k,d_out,M,fmt", [(*s, f) for s in SHAPES for f in FORMATS if f == "u8" or s[0] < 2000])
def test_input_gradient(d_in, k, d_out, M, fmt):
    g, l, D, C = projection(d_in, k, d_out, fmt, M)
    dY = torch.randn(M, d_out, generator=torch.Generator().manual_seed(M)).half().cuda()
    pad = torch.full((M * d_in + 64,), 7.0, dtype=torch.float16, device="cuda")
    dX = pad[:M * d_in].view(M, d_in)
    dp.dictproj_backward_input(dY.data_ptr(), M, l, g, dX.data_ptr(), stream())
    torch.cuda.synchronize()
    check(dX, dY, D, C)
    assert (pad[M * d_in:] == 7).all()
    first = dX.clone()
    dp.dictproj_backward_input(dY.data_ptr(), M, l, g, dX.data_ptr(), stream())
    torch.cuda.synchronize()
    assert torch.equal(first, dX)


def test_input_gradient_agrees_with_the_forward():
    # the adjoint: sum dY * forward(X) = sum X * input gradient(dY), each side with its own roundings
    g, l, D, C = projection(512, 256, 384, "u8", 64)
    X, dY = (torch.randn(64, n, generator=torch.Generator().manual_seed(n)).half().cuda() for n in (512, 384))
    Y, dX = torch.empty(64, 384, dtype=torch.float16, device="cuda"), torch.empty_like(X)
    dp.dictproj_forward(X.data_ptr(), 64, l, g, Y.data_ptr(), stream())
    dp.dictproj_backward_input(dY.data_ptr(), 64, l, g, dX.data_ptr(), stream())
    torch.cuda.synchronize()
    a, b = (dY.double() * Y.double()).sum().item(), (X.double() * dX.double()).sum().item()
    # each side's error is a random sum: two roundings (2^-11 each at most) of 24576 and 32768 products
    size = U16 * 2 * ((dY.double() * Y.double()).norm() + (X.double() * dX.double()).norm()).item()
    assert abs(a - b) <= 4 * size


def test_fewer_rows_captured_and_interleaved_with_the_forward():
    g, l, D, C = projection(256, 128, 264, "u8", 100)
    dY, X = (torch.randn(100, n, generator=torch.Generator().manual_seed(n)).half().cuda() for n in (264, 256))
    dX = torch.full((100, 256), 7.0, dtype=torch.float16, device="cuda")
    Y, Y0 = (torch.empty(100, 264, dtype=torch.float16, device="cuda") for _ in range(2))
    dp.dictproj_forward(X.data_ptr(), 100, l, g, Y0.data_ptr(), stream())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dp.dictproj_forward(X.data_ptr(), 100, l, g, Y.data_ptr(), side.cuda_stream)
        dp.dictproj_backward_input(dY.data_ptr(), 33, l, g, dX.data_ptr(), side.cuda_stream)
        dp.dictproj_forward(X.data_ptr(), 100, l, g, Y.data_ptr(), side.cuda_stream)
    dY.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(dX[:33], dY[:33], D, C)
    assert (dX[33:] == 7).all() and torch.equal(Y, Y0)


def test_refusals_leave_the_output_alone():
    g, l, _, _ = projection(64, 32, 40, "u8", 8)
    bare = dp.dictproj_pack_group(synth.gen_dictionary(41, 0, 0, 64, 32), 8)
    other = dp.dictproj_pack_group(synth.gen_dictionary(41, 0, 0, 64, 48), 8)
    C = synth.gen_coeff(41, 0, 0, 0, 32, 41, 0.3)
    odd = dp.dictproj_pack_layer(C.col_ptr, C.atom_idx, C.vals, 32, 41)
    dp.dictproj_group_reserve_backward(g, 41)
    dY, dX = torch.zeros(16, 64, dtype=torch.float16, device="cuda"), torch.full((16, 64), 7.0, dtype=torch.float16, device="cuda")
    f = lambda y, M, layer, group, x: dp.lib().dictproj_backward_input(y, M, layer.handle, group.handle, x, stream())  # noqa: E731
    y, x = dY.data_ptr(), dX.data_ptr()
    assert f(None, 1, l, g, x) == -1 and f(y, 1, l, g, None) == -1
    assert f(y, 0, l, g, x) == -5 and f(y, 9, l, g, x) == -5
    assert f(y, 1, l, bare, x) == -5  # nothing reserved
    assert f(y, 1, l, other, x) == -4
    assert f(y, 1, odd, g, x) == -2
    assert f(y + 2, 1, l, g, x) == -3 and f(y, 1, l, g, x + 8) == -3
    assert f(x + 16, 8, l, g, x) == -5  # dX over dY
    torch.cuda.synchronize()
    assert (dX == 7).all()
    assert f(y, 8, l, g, x) == 0
