"""Low-rank adapters of many requests beside a projection: forward, gradients, plans and refusals."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import adapter_reference as ref  # noqa: E402
import dictionary_compressed_linear_b200 as dp  # noqa: E402
import synth  # noqa: E402
from gpu_helpers import device_projection, oracle_forward, oracle_projection  # noqa: E402

NAN = float("nan")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def stream():
    return torch.cuda.current_stream().cuda_stream


def ids_of(kind, M, n, seed=1):
    g = np.random.default_rng(seed)
    a = {"one": np.zeros(M, int), "each": np.arange(M) % n, "random": g.integers(0, n, M),
         "some": np.where(g.random(M) < 0.3, -1, g.integers(0, n, M)), "none": np.full(M, -1),
         "last": np.full(M, n - 1), "runs": np.sort(g.integers(0, n, M)),
         # half of the rows in one run of slot 3, the others anywhere (or nowhere)
         "crowd": np.where(np.arange(M) < M // 2, 3, g.integers(-1, n, M)),
         "wild": g.choice([-7, n, n + 5, 2 ** 31 - 1, -2 ** 31, 0, n - 1], M)}[kind]
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def clean(ids, n):
    return torch.where((ids >= 0) & (ids < n), ids, torch.full_like(ids, -1))


def planned(ids, n, max_rows=None):
    r = dp.dictproj_rows_create(max_rows or ids.numel(), n)
    dp.dictproj_rows_set(r, ids.data_ptr(), ids.numel(), stream())
    return r


def normal(*shape, seed=2, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).half().cuda()


CASES = [  # rows, d_in, d_out, max_rank, ranks, ids
    (1, 32, 1, 1, [1], "one"), (1, 4096, 4096, 16, [16], "one"), (3, 64, 7, 3, [3, 2], "random"),
    (8, 256, 264, 16, [16] * 8, "each"), (17, 1376, 1001, 24, [24, 1, 0, 17], "some"),
    (33, 96, 513, 128, [128, 127, 65], "random"), (64, 4096, 11008, 16, [16] * 64, "each"),
    (65, 512, 130, 64, [64, 33], "one"), (100, 1376, 1001, 12, [12, 7, 2, 11], "some"),
    (129, 2048, 72, 32, [32, 31], "last"), (200, 64, 64, 5, [5] * 9, "wild"), (16, 128, 96, 8, [8], "none"),
    (300, 320, 2000, 48, [40, 48, 16], "runs"), (1000, 160, 88, 100, [100, 3], "random"), (15, 11008, 40, 80, [80], "one")]


# batches of many rows: tiles of 64 and 128 rows, runs of rows and scattered ones, slots with many rows beside
# slots with few, every template rank, widths that end inside a block of columns
MANY = [
    (400, 96, 72, 16, [16], "one"), (513, 352, 328, 16, [16, 9, 0], "runs"), (700, 160, 200, 32, [32, 17], "some"),
    (640, 4096, 1000, 32, [20, 32, 1], "random"), (1500, 224, 136, 64, [64, 33], "runs"), (260, 64, 520, 64, [50], "last"),
    (900, 288, 1096, 128, [128, 40], "random"), (777, 544, 776, 128, [100, 65, 3], "runs"), (1030, 128, 77, 16, [16, 5], "runs"),
    (600, 192, 129, 64, [64, 30], "some"), (520, 96, 264, 32, [24] * 40, "crowd"), (1100, 160, 96, 96, [96] * 60, "crowd"),
    (600, 64, 75, 16, [16] * 50, "crowd"), (300, 64, 64, 16, [16, 8], "none"), (2048, 64, 64, 8, [8] * 9, "wild")]


@pytest.mark.parametrize("M,d_in,d_out,R,ranks,kind", CASES + MANY)
@pytest.mark.parametrize("mode", ["apart", "in place", "zero"])
def test_forward(M, d_in, d_out, R, ranks, kind, mode):
    pool = ref.Pool(d_in, d_out, R, ranks, seed=M)
    ids = ids_of(kind, M, len(ranks))
    X, base = normal(M, d_in), normal(M, d_out, seed=3)
    h, rows = pool.upload(dp, M, stream()), planned(ids, len(ranks))
    want, W = ref.forward(pool, clean(ids, len(ranks)), X, None if mode == "zero" else base)
    Y = base.clone() if mode == "in place" else torch.full_like(base, NAN)
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), {"apart": base, "in place": Y}.get(mode, None).data_ptr() if mode != "zero" else 0,
                                Y.data_ptr(), stream())
    torch.cuda.synchronize()
    ref.assert_half(Y, want, W, d_in + R, mode)


@pytest.mark.parametrize("M,d_in,d_out,R,ranks,kind", CASES + MANY)
def test_backward(M, d_in, d_out, R, ranks, kind):
    pool = ref.Pool(d_in, d_out, R, ranks, seed=M)
    n = len(ranks)
    ids = ids_of(kind, M, n)
    X, dY, base = normal(M, d_in), normal(M, d_out, seed=3, scale=0.05), normal(M, d_in, seed=4)
    h, rows = pool.upload(dp, M, stream()), planned(ids, n)
    w = ref.backward(pool, clean(ids, n), X, dY, base)
    dX = torch.full_like(X, NAN)
    dA, dB = torch.full((n, R, d_in), NAN, device="cuda"), torch.full((n, R, d_out), NAN, device="cuda")
    call = lambda acc: dp.dictproj_adapter_backward(  # noqa: E731
        h, rows, X.data_ptr(), dY.data_ptr(), base.data_ptr(), dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), acc, stream())
    call(False)
    torch.cuda.synchronize()
    ref.assert_half(dX, w["dX"], w["WX"], d_out + R, "dX")
    ref.assert_float(dA, w["dA"], w["WA"], d_out + M, "dA")
    ref.assert_float(dB, w["dB"], w["WB"], d_in + M, "dB")
    first = dX.clone(), dA.clone(), dB.clone()
    call(False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (dX, dA, dB)))  # the same bits
    call(True)
    torch.cuda.synchronize()
    assert torch.equal(dA, first[1] + first[1]) and torch.equal(dB, first[2] + first[2])


def test_backward_of_parts_only():
    pool = ref.Pool(256, 200, 16, [16, 9], seed=1)
    ids = ids_of("some", 90, 2)
    X, dY = normal(90, 256), normal(90, 200, seed=3)
    h, rows = pool.upload(dp, 90, stream()), planned(ids, 2)
    w = ref.backward(pool, ids, X, dY)
    dX = torch.full_like(X, NAN)
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, dX.data_ptr(), 0, 0, False, stream())
    ref.assert_half(dX, w["dX"], w["WX"], 216, "dX alone")
    dA, dB = torch.full((2, 16, 256), NAN, device="cuda"), torch.full((2, 16, 200), NAN, device="cuda")
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, 0, dA.data_ptr(), dB.data_ptr(), False, stream())
    ref.assert_float(dA, w["dA"], w["WA"], 290, "dA")
    ref.assert_float(dB, w["dB"], w["WB"], 346, "dB")
    acc = X.clone()
    dp.dictproj_adapter_backward(h, rows, X.clone().data_ptr(), dY.data_ptr(), acc.data_ptr(), acc.data_ptr(), 0, 0, False, stream())
    torch.cuda.synchronize()
    w = ref.backward(pool, ids, X, dY, X)
    ref.assert_half(acc, w["dX"], w["WX"], 216, "dX in place")


def test_gradients_agree_with_differences():
    # L(A, B, X) = sum G * Y in fp64; a central difference along a random direction is exact up to rounding
    # (L is at most quadratic along it), so it is off by fp64's 2^-53 / h of the terms alone.
    pool = ref.Pool(96, 80, 8, [8, 5], seed=3)
    ids = ids_of("random", 40, 2)
    X, G = normal(40, 96), normal(40, 80, seed=5)
    h, rows = pool.upload(dp, 40, stream()), planned(ids, 2)
    dX = torch.empty_like(X)
    dA, dB = torch.empty(2, 8, 96, device="cuda"), torch.empty(2, 8, 80, device="cuda")
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), G.data_ptr(), 0, dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()

    def loss(A, B, x):
        total = 0.0
        for s in range(2):
            at = ref.rows_of(ids, s)
            total = total + pool.scale[s] * (((x[at] @ A[s].T) @ B[s]) * G[at].double()).sum()
        return total

    A, B, x = [a.double() for a in pool.A], [b.double() for b in pool.B], X.double()
    g = torch.Generator(device="cuda").manual_seed(7)
    eA, eB = ([torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64) for w in ws] for ws in (A, B))
    eX, step = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64), 1e-3
    move = lambda ws, es, k: [w + k * step * e for w, e in zip(ws, es)]  # noqa: E731
    for got, plus, minus in (
            (sum((dA[s, :r].double() * eA[s]).sum() for s, r in enumerate(pool.ranks)), loss(move(A, eA, 1), B, x), loss(move(A, eA, -1), B, x)),
            (sum((dB[s, :r].double() * eB[s]).sum() for s, r in enumerate(pool.ranks)), loss(A, move(B, eB, 1), x), loss(A, move(B, eB, -1), x)),
            ((dX.double() * eX).sum(), loss(A, B, x + step * eX), loss(A, B, x - step * eX))):
        want = ((plus - minus) / (2 * step)).item()
        # the fp16 rounding of dX is 2^-11 an element at most, and random over 3840 of them
        size = (dX.double().norm() * ref.U16).item()
        assert abs(got.item() - want) <= 4 * size + 1e-4 * abs(want)


def test_rows_without_an_adapter_and_foreign_values_stay_apart():
    pool = ref.Pool(128, 96, 8, [8, 8], seed=2)
    ids = torch.tensor([0, -1, 1, 0, 5, 1, 0, -1], dtype=torch.int32, device="cuda")
    X, base = normal(8, 128), normal(8, 96, seed=3)
    X[1] = NAN  # a row without an adapter is not read
    X[3, 5] = float("inf")  # reaches its own row alone
    base[4] = NAN
    h, rows = pool.upload(dp, 8, stream()), planned(ids, 2)
    Y = base.clone()
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), Y.data_ptr(), Y.data_ptr(), stream())
    torch.cuda.synchronize()
    assert torch.equal(Y[1].view(torch.int16), base[1].view(torch.int16)) and torch.equal(Y[4].view(torch.int16), base[4].view(torch.int16))
    assert not torch.isfinite(Y[3]).any()
    keep = [0, 2, 5, 6]
    Z = X.clone()
    Z[1], Z[3] = 0, 0
    want, W = ref.forward(pool, clean(ids, 2), Z, base)
    ref.assert_half(Y[keep], want[keep], W[keep], 136)
    dA, dB = torch.empty(2, 8, 128, device="cuda"), torch.empty(2, 8, 96, device="cuda")
    dY = base.clone()
    dY[1] = NAN
    X[3, 5] = 1.0
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, 0, dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    assert torch.isfinite(dA).all() and torch.isfinite(dB).all()


@pytest.mark.parametrize("d_out", [96, 75])
@pytest.mark.parametrize("order", ["runs", "scattered"])
def test_many_rows_keep_foreign_values_apart(order, d_out):
    # slot 0 ends inside a tile; behind it lie rows of slot 1 and of none, full of infinities and NaN
    M, n0 = 600, 300
    pool = ref.Pool(128, d_out, 16, [16, 16], seed=2)
    ids = torch.tensor([0] * n0 + [1] * 200 + [-1] * 100, dtype=torch.int32, device="cuda")
    if order == "scattered":
        ids = ids[torch.randperm(M, generator=torch.Generator().manual_seed(1)).cuda()]
    X, dY, base = normal(M, 128), normal(M, d_out, seed=3), normal(M, d_out, seed=4)
    X[ids != 0], dY[ids != 0] = float("inf"), NAN
    mine = ids == 0
    h, rows = pool.upload(dp, M, stream()), planned(ids, 2)
    Y, dX = base.clone(), torch.zeros_like(X)
    dA, dB = torch.empty(2, 16, 128, device="cuda"), torch.empty(2, 16, d_out, device="cuda")
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), Y.data_ptr(), Y.data_ptr(), stream())
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    one = ref.Pool(128, d_out, 16, [16], seed=2)
    one.A, one.B, one.scale = pool.A[:1], pool.B[:1], pool.scale[:1]
    own = ids[mine]
    want, W = ref.forward(one, own, X[mine], base[mine])
    ref.assert_half(Y[mine], want, W, 144)
    assert torch.equal(Y[ids == -1], base[ids == -1])
    w = ref.backward(one, own, X[mine], dY[mine])
    ref.assert_half(dX[mine], w["dX"], w["WX"], d_out + 16)
    ref.assert_float(dA[:1], w["dA"], w["WA"], d_out + n0)
    ref.assert_float(dB[:1], w["dB"], w["WB"], 128 + n0)
    assert (dX[ids == -1] == 0).all()


def test_two_pools_on_two_streams_at_once():
    # nothing is shared between pools: their workspaces are their own
    work = []
    for k, (M, d_out) in enumerate(((1024, 512), (700, 264))):
        pool = ref.Pool(256, d_out, 32, [32, 20], seed=k)
        ids, X, dY = ids_of("runs", M, 2, seed=k), normal(M, 256, seed=k), normal(M, d_out, seed=k + 5)
        work.append(dict(pool=pool, ids=ids, X=X, dY=dY, h=pool.upload(dp, M, stream()), rows=planned(ids, 2), s=torch.cuda.Stream(),
                         Y=torch.empty(M, d_out, dtype=torch.float16, device="cuda"), dX=torch.empty_like(X),
                         dA=torch.empty(2, 32, 256, device="cuda"), dB=torch.empty(2, 32, d_out, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for w in work:
            s = w["s"].cuda_stream
            dp.dictproj_adapter_forward(w["h"], w["rows"], w["X"].data_ptr(), 0, w["Y"].data_ptr(), s)
            dp.dictproj_adapter_backward(w["h"], w["rows"], w["X"].data_ptr(), w["dY"].data_ptr(), 0, w["dX"].data_ptr(),
                                         w["dA"].data_ptr(), w["dB"].data_ptr(), False, s)
    torch.cuda.synchronize()
    for w in work:
        want, W = ref.forward(w["pool"], w["ids"], w["X"])
        ref.assert_half(w["Y"], want, W, 288)
        b = ref.backward(w["pool"], w["ids"], w["X"], w["dY"])
        n = w["dY"].shape
        ref.assert_half(w["dX"], b["dX"], b["WX"], n[1] + 32)
        ref.assert_float(w["dA"], b["dA"], b["WA"], n[1] + n[0])
        ref.assert_float(w["dB"], b["dB"], b["WB"], 256 + n[0])
    assert dp.dictproj_check_status(stream()) == 0


@pytest.mark.parametrize("M,R", [(2048, 16), (1024, 64), (300, 128)])
def test_long_sums_keep_the_accuracy_of_fp32(M, R):
    # The tensor cores sum runs of at most 8 steps (128 columns, or a 64-row tile in two parts) on their own,
    # 2^-23 of the run a step at most; the runs' sums are fp32 additions, 2^-24 each at random over some 150 of them.
    pool = ref.Pool(4096, 1024, R, [R], seed=4)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    X, dY = normal(M, 4096), normal(M, 1024, seed=3)
    h, rows = pool.upload(dp, M, stream()), planned(ids, 1)
    dA, dB = torch.empty(1, R, 4096, device="cuda"), torch.empty(1, R, 1024, device="cuda")
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, 0, dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    w = ref.backward(pool, ids, X, dY)
    limit = 8 * 2.0 ** -23 + 2.0 ** -24 * 150 ** 0.5
    for got, want in ((dA, w["dA"]), (dB, w["dB"])):
        assert ((got.double() - want).norm() / want.norm()).item() <= limit


@pytest.mark.parametrize("M,d_in,d_out,R", [(1300, 4096, 1025, 16), (300, 4096, 1024, 16), (520, 2048, 2047, 64), (16, 4096, 4096, 16), (12, 4096, 1001, 128)])
def test_long_sums_of_the_other_kernels_keep_the_accuracy_of_fp32(M, d_in, d_out, R):
    # as above, for rows on mma.sync (any width, or too few rows for tcgen05) and for few rows (fp32 throughout)
    pool = ref.Pool(d_in, d_out, R, [R], seed=4)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    X, dY = normal(M, d_in), normal(M, d_out, seed=3)
    h, rows = pool.upload(dp, M, stream()), planned(ids, 1)
    dA, dB = torch.empty(1, R, d_in, device="cuda"), torch.empty(1, R, d_out, device="cuda")
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, 0, dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    w = ref.backward(pool, ids, X, dY)
    limit = 8 * 2.0 ** -23 + 2.0 ** -24 * 150 ** 0.5
    for got, want in ((dA, w["dA"]), (dB, w["dB"])):
        assert ((got.double() - want).norm() / want.norm()).item() <= limit


@pytest.mark.parametrize("M", [12, 600])
@pytest.mark.parametrize("d_out", [96, 75])
@pytest.mark.parametrize("mode", ["zero", "apart", "in place"])
def test_every_row_of_dx_is_written(M, d_out, mode):
    # rows of foreign slots are full of infinities and NaN, those without an adapter get base, or zeros
    pool = ref.Pool(128, d_out, 16, [16, 16], seed=2)
    ids = ids_of("some", M, 2, seed=5)
    X, dY, base = normal(M, 128), normal(M, d_out, seed=3), normal(M, 128, seed=4)
    X[ids != 0], dY[ids != 0] = float("inf"), NAN
    h, rows = pool.upload(dp, M, stream()), planned(ids, 2)
    for grads in (False, True):
        dX = base.clone() if mode == "in place" else torch.full_like(base, NAN)
        dA, dB = torch.empty(2, 16, 128, device="cuda"), torch.empty(2, 16, d_out, device="cuda")
        dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), {"zero": 0, "apart": base.data_ptr(), "in place": dX.data_ptr()}[mode],
                                     dX.data_ptr(), dA.data_ptr() if grads else 0, dB.data_ptr() if grads else 0, False, stream())
        torch.cuda.synchronize()
        none = ids == -1
        assert none.any() and torch.equal(dX[none], torch.zeros_like(dX[none]) if mode == "zero" else base[none])
        mine = ids == 0
        one = ref.Pool(128, d_out, 16, [16], seed=2)
        one.A, one.B, one.scale = pool.A[:1], pool.B[:1], pool.scale[:1]
        w = ref.backward(one, ids[mine], X[mine], dY[mine], None if mode == "zero" else base[mine])
        ref.assert_half(dX[mine], w["dX"], w["WX"], d_out + 16)


@pytest.mark.parametrize("size", [1e-7, 1e4])
def test_small_and_large_activations_keep_their_digits(size):
    # T is far outside fp16's comfortable range: small gradients must not fall to zero in a sum
    pool = ref.Pool(512, 256, 16, [16, 16], seed=4)
    ids = ids_of("random", 70, 2)
    X, dY = normal(70, 512), normal(70, 256, seed=3, scale=size)
    h, rows = pool.upload(dp, 70, stream()), planned(ids, 2)
    dA, dB = torch.empty(2, 16, 512, device="cuda"), torch.empty(2, 16, 256, device="cuda")
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, 0, dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    w = ref.backward(pool, ids, X, dY)
    ref.assert_float(dA, w["dA"], w["WA"], 256 + 70)
    ref.assert_float(dB, w["dB"], w["WB"], 512 + 70)


@pytest.mark.parametrize("M,d_out,R", [(16, 96, 16), (300, 77, 16), (300, 1001, 64), (700, 96, 16), (700, 264, 32), (300, 1024, 64), (300, 1024, 128)])
def test_ranks_of_different_size_keep_their_digits(M, d_out, R):
    # 2^26 between the first rank's weights and the last one's: every rank's gradients are as exact as they would
    # be alone. Bound as for the long sums, and T in two parts, 2^-22 of it.
    pool = ref.Pool(512, d_out, R, [R], seed=4)
    size = 2.0 ** (10 - 26 * torch.arange(R, device="cuda") / (R - 1))[:, None]
    g = torch.Generator(device="cuda").manual_seed(5)
    pool.A, pool.B = ([(torch.randn(R, n, generator=g, device="cuda") * size).half()] for n in (512, d_out))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    X, dY = normal(M, 512), normal(M, d_out, seed=3, scale=0.05)
    h, rows = pool.upload(dp, M, stream()), planned(ids, 1)
    dA, dB = torch.empty(1, R, 512, device="cuda"), torch.empty(1, R, d_out, device="cuda")
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, 0, dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    w = ref.backward(pool, ids, X, dY)
    limit = 8 * 2.0 ** -23 + 2.0 ** -24 * 150 ** 0.5 + 2.0 ** -22
    for got, want in ((dA, w["dA"]), (dB, w["dB"])):
        off = (got.double() - want).norm(dim=2) / want.norm(dim=2)
        assert off.max().item() <= limit, (off.argmax().item(), off.max().item())


@pytest.mark.parametrize("M,d_out,R", [(40, 96, 16), (300, 77, 16), (300, 1001, 64), (600, 96, 16), (700, 264, 32), (300, 1024, 128)])
def test_rows_of_different_size_keep_their_digits(M, d_out, R):
    # rows of 2^13 and of 2^-17 in turn: the small ones' results are rounded once, as if they were alone
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    size = torch.where(torch.arange(M, device="cuda") % 2 == 0, 2.0 ** -17, 2.0 ** 13)[:, None]
    g = torch.Generator(device="cuda").manual_seed(5)
    X, dY = ((torch.randn(M, n, generator=g, device="cuda") * size).half() for n in (512, d_out))
    rows = planned(ids, 1)
    pool = ref.Pool(512, d_out, R, [R], seed=4)
    pool.B = [(torch.randn(R, d_out, generator=g, device="cuda") * 2.0 ** 8).half()]
    Y = torch.full_like(dY, NAN)
    dp.dictproj_adapter_forward(pool.upload(dp, M, stream()), rows, X.data_ptr(), 0, Y.data_ptr(), stream())
    torch.cuda.synchronize()
    want, W = ref.forward(pool, ids, X)
    ref.assert_half(Y[::2], want[::2], W[::2], 512 + R, "Y")
    pool = ref.Pool(512, d_out, R, [R], seed=4)
    pool.A = [(torch.randn(R, 512, generator=g, device="cuda") * 2.0 ** 8).half()]
    h = pool.upload(dp, M, stream())
    for grads in (False, True):
        dX = torch.full_like(X, NAN)
        dA, dB = torch.empty(1, R, 512, device="cuda"), torch.empty(1, R, d_out, device="cuda")
        dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, dX.data_ptr(), dA.data_ptr() if grads else 0,
                                     dB.data_ptr() if grads else 0, False, stream())
        torch.cuda.synchronize()
        w = ref.backward(pool, ids, X, dY)
        ref.assert_half(dX[::2], w["dX"][::2], w["WX"][::2], d_out + R, "dX")


@pytest.mark.parametrize("M", [256, 511, 2048, 4096])
@pytest.mark.parametrize("slots,used,R", [(64, 1, 16), (64, 4, 16), (64, 2, 64), (9, 1, 32), (1024, 3, 16)])
def test_large_pools_of_which_a_batch_uses_few(M, slots, used, R):
    # the kernels are chosen by the pool's slots; the others' gradients are zeros
    at = np.linspace(0, slots - 1, used).astype(int)  # the first slot and the last among them
    ranks = [0] * slots
    for i, s in enumerate(at):
        ranks[s] = R - i
    pool = ref.Pool(160, 96, R, ranks, seed=M)
    ids = torch.tensor(np.repeat(at, -(-M // used))[:M], dtype=torch.int32, device="cuda")
    X, dY, base = normal(M, 160), normal(M, 96, seed=3, scale=0.05), normal(M, 96, seed=4)
    h, rows = pool.upload(dp, M, stream()), planned(ids, slots)
    Y, dX = torch.full_like(base, NAN), torch.full_like(X, NAN)
    dA, dB = torch.full((slots, R, 160), NAN, device="cuda"), torch.full((slots, R, 96), NAN, device="cuda")
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), base.data_ptr(), Y.data_ptr(), stream())
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), False, stream())
    torch.cuda.synchronize()
    want, W = ref.forward(pool, ids, X, base)
    ref.assert_half(Y, want, W, 160 + R)
    w = ref.backward(pool, ids, X, dY)
    ref.assert_half(dX, w["dX"], w["WX"], 96 + R)
    ref.assert_float(dA, w["dA"], w["WA"], 96 + M)
    ref.assert_float(dB, w["dB"], w["WB"], 160 + M)


def test_a_slot_is_replaced_and_emptied():
    pool, other = ref.Pool(64, 41, 24, [24, 20], seed=1), ref.Pool(64, 41, 24, [3, 24], seed=9)
    ids, X = ids_of("each", 6, 2), normal(6, 64)
    h, rows = pool.upload(dp, 6, stream()), planned(ids, 2)
    dp.dictproj_adapters_set(h, 0, 3, other.scale[0], other.A[0].data_ptr(), other.B[0].data_ptr(), stream())
    dp.dictproj_adapters_set(h, 1, 0, 0.0, 0, 0, stream())
    Y = torch.full((6, 41), NAN, dtype=torch.float16, device="cuda")
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), 0, Y.data_ptr(), stream())
    torch.cuda.synchronize()
    other.ranks = [3, 0]
    want, W = ref.forward(other, ids, X)
    ref.assert_half(Y, want, W, 88)
    assert (Y[1::2] == 0).all()


def test_many_slots_and_offsets_past_32_bits():
    n, d_in, d_out = 1024, 4096, 96  # the pool's A alone has 2^30 bytes and more
    h = dp.dictproj_adapters_create(d_in, d_out, 128, n, 2048)
    pool = ref.Pool(d_in, d_out, 128, [0] * (n - 2) + [128, 77], seed=6)
    for s in (n - 2, n - 1):
        dp.dictproj_adapters_set(h, s, pool.ranks[s], pool.scale[s], pool.A[s].data_ptr(), pool.B[s].data_ptr(), stream())
    ids = torch.arange(2048, device="cuda").remainder(n).to(torch.int32)
    X, rows = normal(2048, d_in), planned(ids, n)
    Y = torch.full((2048, d_out), NAN, dtype=torch.float16, device="cuda")
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), 0, Y.data_ptr(), stream())
    torch.cuda.synchronize()
    want, W = ref.forward(pool, ids, X)
    ref.assert_half(Y, want, W, d_in + 128)
    h.free()
    M, d_out = 400_000, 11008  # Y has 4.4e9 elements
    pool = ref.Pool(32, d_out, 1, [1], seed=6)
    h = pool.upload(dp, M, stream())
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[[5, M // 2, M - 1]] = 0
    X, rows = normal(8, 32).repeat(M // 8, 1), planned(ids, 1)
    Y = torch.full((M, d_out), 3.0, dtype=torch.float16, device="cuda")
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), Y.data_ptr(), Y.data_ptr(), stream())
    torch.cuda.synchronize()
    at = [4, 5, M // 2, M - 2, M - 1]
    want, W = ref.forward(pool, ids[at], X[at], torch.full((5, d_out), 3.0, dtype=torch.float16, device="cuda"))
    ref.assert_half(Y[at], want, W, 33)


@pytest.mark.parametrize("M", [20, 600])
def test_captured_calls_plan_anew_and_other_streams(M):
    pool = ref.Pool(256, 264, 16, [16, 8, 4], seed=2)
    h = pool.upload(dp, M, stream())
    ids, X = ids_of("random", M, 3), normal(M, 256)
    rows = dp.dictproj_rows_create(M, 3)
    Y, dX = torch.zeros(M, 264, dtype=torch.float16, device="cuda"), torch.zeros_like(X)
    dY = normal(M, 264, seed=8)
    dA, dB = torch.zeros(3, 16, 256, device="cuda"), torch.zeros(3, 16, 264, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(s):
        dp.dictproj_rows_set(rows, ids.data_ptr(), M, s)
        dp.dictproj_adapter_forward(h, rows, X.data_ptr(), 0, Y.data_ptr(), s)
        dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), False, s)

    with torch.cuda.stream(side):
        step(side.cuda_stream)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side.cuda_stream)
    for seed in (3, 4):
        ids.copy_(ids_of("some", M, 3, seed=seed))
        X.copy_(normal(M, 256, seed=seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, W = ref.forward(pool, ids, X)
        ref.assert_half(Y, want, W, 272)
        w = ref.backward(pool, ids, X, dY)
        ref.assert_half(dX, w["dX"], w["WX"], 280)
        ref.assert_float(dA, w["dA"], w["WA"], 264 + M)
        ref.assert_float(dB, w["dB"], w["WB"], 256 + M)


@pytest.mark.parametrize("M", [8, 300, 700])
@pytest.mark.parametrize("slots", [1, 3])
def test_a_captured_call_takes_no_plan_of_more_rows(M, slots):
    # the arrays hold twice the rows, so that only the kernels' own check is tested
    pool = ref.Pool(256, 264, 16, [16, 8, 4][:slots], seed=2)
    h = pool.upload(dp, 2 * M, stream())
    rows = dp.dictproj_rows_create(2 * M, slots)
    ids, X, dY = ids_of("each", 2 * M, slots), normal(2 * M, 256), normal(2 * M, 264, seed=8)
    Y, dX = torch.zeros_like(dY), torch.zeros_like(X)
    dA, dB = torch.zeros(slots, 16, 256, device="cuda"), torch.zeros(slots, 16, 264, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dp.dictproj_rows_set(rows, ids.data_ptr(), M, side.cuda_stream)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dp.dictproj_adapter_forward(h, rows, X.data_ptr(), 0, Y.data_ptr(), side.cuda_stream)
        dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), 0, dX.data_ptr(), dA.data_ptr(), dB.data_ptr(), False,
                                     side.cuda_stream)
    outs = (Y, dX, dA, dB)
    for planned_rows in (M, 2 * M, M - 3):  # as captured, more, fewer
        for t in outs:
            t.fill_(7)
        dp.dictproj_rows_set(rows, ids.data_ptr(), planned_rows, stream())
        graph.replay()
        torch.cuda.synchronize()
        if planned_rows > M:
            assert (Y == 7).all() and (dX == 7).all()
            assert ((dA == 7) | (dA == 0)).all() and ((dB == 7) | (dB == 0)).all()
            continue
        n = planned_rows
        want, W = ref.forward(pool, ids[:n], X[:n])
        ref.assert_half(Y[:n], want, W, 272)
        w = ref.backward(pool, ids[:n], X[:n], dY[:n])
        ref.assert_half(dX[:n], w["dX"], w["WX"], 280)
        ref.assert_float(dA, w["dA"], w["WA"], 264 + M)
        ref.assert_float(dB, w["dB"], w["WB"], 256 + M)
        assert (Y[n:] == 7).all() and (dX[n:] == 7).all()


def test_a_plan_that_was_only_captured_has_no_rows():
    pool = ref.Pool(256, 264, 16, [16, 8], seed=2)
    h = pool.upload(dp, 8, stream())
    rows = dp.dictproj_rows_create(8, 2)
    ids, X = ids_of("each", 8, 2), normal(8, 256)
    Y = torch.full((8, 264), 7.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.dictproj_rows_set(rows, ids.data_ptr(), 8, stream())
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), 0, Y.data_ptr(), stream())
    torch.cuda.synchronize()
    assert (Y == 7).all()
    graph.replay()
    dp.dictproj_adapter_forward(h, rows, X.data_ptr(), 0, Y.data_ptr(), stream())
    torch.cuda.synchronize()
    want, W = ref.forward(pool, ids, X)
    ref.assert_half(Y, want, W, 272)


def _projection(d_in, d_out, k, M, seed=30):
    D, C = synth.gen_dictionary(seed, 0, 0, d_in, k), synth.gen_coeff(seed, 0, 0, 0, k, d_out, 0.4)
    g, l = device_projection(D, C, M)
    return g, l, oracle_projection(D, C)


@pytest.mark.parametrize("M", [1, 5, 40])
def test_projection_with_adapters(M):
    g, l, packed = _projection(256, 200, 128, M)
    pool = ref.Pool(256, 200, 16, [16, 7], seed=5)
    ids, X = ids_of("some", M, 2, seed=M), normal(M, 256)
    h, rows = pool.upload(dp, M, stream()), planned(ids, 2)
    Y, P = (torch.full((M, 200), NAN, dtype=torch.float16, device="cuda") for _ in range(2))
    dp.dictproj_forward_adapters(X.data_ptr(), l, g, h, rows, Y.data_ptr(), stream())
    dp.dictproj_forward(X.data_ptr(), M, l, g, P.data_ptr(), stream())
    torch.cuda.synchronize()
    want, W = ref.forward(pool, ids, X, P)  # the projection itself is held to the oracle elsewhere
    ref.assert_half(Y, want, W, 272)
    exact = torch.tensor(oracle_forward(X.cpu().numpy(), *packed), device="cuda")
    whole, _ = ref.forward(pool, ids, X, exact)
    assert ((Y.double() - whole).norm() / whole.norm()).item() <= 5e-3  # the projection's own tolerance


def test_refusals_leave_the_outputs_alone():
    pool = ref.Pool(64, 48, 8, [8, 4], seed=1)
    h = pool.upload(dp, 4, stream())
    ids = ids_of("each", 4, 2)
    rows, empty = planned(ids, 2), dp.dictproj_rows_create(4, 2)
    long, wide = planned(ids_of("each", 5, 2), 2), planned(ids, 3)
    X, Y = normal(8, 64), torch.full((8, 64), 7.0, dtype=torch.float16, device="cuda")
    dA, dB = torch.full((2, 8, 64), 7.0, device="cuda"), torch.full((2, 8, 48), 7.0, device="cuda")
    L, s, x, y = dp.lib(), stream(), X.data_ptr(), Y.data_ptr()
    fwd = lambda *a: L.dictproj_adapter_forward(*a, s)  # noqa: E731
    assert fwd(h.handle, empty.handle, x, None, y) == -5  # nothing planned
    assert fwd(h.handle, long.handle, x, None, y) == -5  # more rows than max_tokens
    assert fwd(h.handle, wide.handle, x, None, y) == -5  # another number of slots
    assert fwd(h.handle, rows.handle, None, None, y) == -1
    assert fwd(h.handle, rows.handle, x + 2, None, y) == -3
    assert fwd(h.handle, rows.handle, x, y + 4, y) == -3
    assert fwd(h.handle, rows.handle, x, None, x + 16) == -5  # Y over X
    assert fwd(h.handle, rows.handle, x, y + 16, y) == -5  # Y over part of base
    back = lambda *a: L.dictproj_adapter_backward(h.handle, rows.handle, *a, 0, s)  # noqa: E731
    assert back(x, y, None, x, None, None) == -5  # dX over X
    assert back(x, y, None, None, dA.data_ptr(), dA.data_ptr()) == -5
    assert back(x, y, None, None, dA.data_ptr(), None) == -1
    assert back(x, y, None, None, dA.data_ptr() + 4, dB.data_ptr()) == -3
    assert back(x, y, None, None, None, None) == -1
    assert L.dictproj_adapters_set(h.handle, 2, 4, 1.0, x, x, s) == -5
    assert L.dictproj_adapters_set(h.handle, 0, 9, 1.0, x, x, s) == -5
    assert L.dictproj_adapters_set(h.handle, 0, 4, float("inf"), x, x, s) == -10
    assert L.dictproj_adapters_set(h.handle, 0, 4, 1.0, x + 1, x, s) == -3
    assert L.dictproj_adapters_set(h.handle, 0, 4, 1.0, None, x, s) == -1
    assert L.dictproj_rows_set(rows.handle, ids.data_ptr(), 5, s) == -5
    assert L.dictproj_rows_set(rows.handle, ids.data_ptr(), 0, s) == -5
    assert L.dictproj_rows_set(rows.handle, ids.data_ptr() + 2, 3, s) == -3
    g, l, _ = _projection(64, 32, 32, 4)
    assert L.dictproj_forward_adapters(x, l.handle, g.handle, h.handle, rows.handle, y, s) == -4  # d_out differs
    torch.cuda.synchronize()
    assert (Y == 7).all() and (dA == 7).all() and (dB == 7).all()
    want, W = ref.forward(pool, ids, X[:4])
    out = torch.empty(4, 48, dtype=torch.float16, device="cuda")
    assert fwd(h.handle, rows.handle, x, None, out.data_ptr()) == 0  # the refused slots kept their weights
    ref.assert_half(out, want, W, 72)


def test_a_training_step_and_the_serving_of_its_result():
    # forward, loss gradient, both backward calls and the optimiser, as a fine-tune runs them
    M, d_in, d_out, r, lr = 48, 256, 192, 8, 1e-3
    g, l, (pd, pc) = _projection(d_in, d_out, 128, M)
    dp.dictproj_group_reserve_backward(g, d_out)
    pool = ref.Pool(d_in, d_out, r, [r, r], seed=5, scale=2.0)
    h = pool.upload(dp, M, stream())
    ids, X, target = ids_of("random", M, 2), normal(M, d_in), normal(M, d_out, seed=6)
    rows = planned(ids, 2)
    master = {n: torch.stack(w).float() for n, w in (("A", pool.A), ("B", pool.B))}
    grad = {n: torch.empty_like(w) for n, w in master.items()}
    state = {n: [torch.zeros_like(w) for _ in range(2)] for n, w in master.items()}
    where = [dp.dictproj_adapters_slot(h, s) for s in range(2)]
    table = [{"p": master[n][s].data_ptr(), "g": grad[n][s].data_ptr(), "m": state[n][0][s].data_ptr(),
              "v": state[n][1][s].data_ptr(), "copy": where[s][n], "n": master[n][s].numel()} for n in "AB" for s in range(2)]
    plan = dp.dictproj_adamw_create(table, 32)
    Y, dX = torch.empty(M, d_out, dtype=torch.float16, device="cuda"), torch.empty_like(X)
    dp.dictproj_forward_adapters(X.data_ptr(), l, g, h, rows, Y.data_ptr(), stream())
    dY = (Y.float() - target.float()).half()
    dp.dictproj_backward_input(dY.data_ptr(), M, l, g, dX.data_ptr(), stream())
    through = dX.clone()
    dp.dictproj_adapter_backward(h, rows, X.data_ptr(), dY.data_ptr(), dX.data_ptr(), dX.data_ptr(), grad["A"].data_ptr(),
                                 grad["B"].data_ptr(), False, stream())
    before = {n: w.double() for n, w in master.items()}
    dp.dictproj_adamw_step(plan, 1, lr, 0.9, 0.999, 1e-8, 0.0, 1.0, stream())
    dp.dictproj_forward_adapters(X.data_ptr(), l, g, h, rows, Y.data_ptr(), stream())
    torch.cuda.synchronize()
    w = ref.backward(pool, ids, X, dY, through)
    ref.assert_half(dX, w["dX"], w["WX"], d_out + r)
    for n in "AB":
        ref.assert_float(grad[n], w["d" + n], w["W" + n], max(d_in, d_out) + M, n)
        # the first step moves every weight by lr against its gradient's sign (m / sqrt(v) = sign but for eps)
        moved = (master[n].double() - before[n]) / lr
        sure = grad[n].abs() > 1e-4
        assert ((moved + grad[n].sign())[sure].abs() <= 2e-4 + 2.0 ** -23 * before[n].abs()[sure] / lr).all()
    pool.A, pool.B = list(master["A"].half()), list(master["B"].half())  # the working copies in the slots
    P = torch.empty_like(Y)
    dp.dictproj_forward(X.data_ptr(), M, l, g, P.data_ptr(), stream())
    torch.cuda.synchronize()
    want, W = ref.forward(pool, ids, X, P)
    ref.assert_half(Y, want, W, d_in + r, "served after the step")


@pytest.mark.parametrize("kind", ["alloc", "copy"])
def test_injected_host_faults_leave_nothing_allocated(kind):
    code = (
        "import torch, dictionary_compressed_linear_b200 as dp\n"
        "x = torch.zeros(1 << 20, device='cuda')\n"
        "import os; os.environ['DICTPROJ_FAULT'] = ''\n"
        "free0 = torch.cuda.mem_get_info()[0]\n"
        f"os.environ['DICTPROJ_FAULT'] = '{kind}'\n"
        # addresses alone: no step is made of them
        "t = [{'n': 1 << 20, **{k: (1 << 40) + (4 * i + j << 22) for j, k in enumerate('pgmv')}} for i in range(500)]\n"
        "calls = {'adamw': lambda: dp.dictproj_adamw_create(t, 32)}\n"
        f"if '{kind}' == 'alloc':\n"
        "    calls.update(pool=lambda: dp.dictproj_adapters_create(4096, 11008, 64, 64, 2048),\n"
        "                 rows=lambda: dp.dictproj_rows_create(1 << 20, 1024))\n"
        f"want = {{'alloc': -7, 'copy': -6}}['{kind}']\n"
        "for name, call in calls.items():\n"
        "    for _ in range(20):\n"
        "        try:\n"
        "            call()\n"
        "            raise SystemExit('no error from ' + name)\n"
        "        except dp.DictprojError as e:\n"
        "            assert e.status == want, (name, e)\n"
        "free1 = torch.cuda.mem_get_info()[0]\n"
        "assert free0 - free1 < 32 << 20, (free0, free1)\n"
        "print('ok')\n")
    env = dict(os.environ, DICTPROJ_FAULT="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


def test_a_wait_that_gives_up_is_reported_by_every_kernel_file():
    dp.dictproj_selftest_wait_timeout(100000, stream())
    assert dp.dictproj_check_status(stream()) == -8
    assert dp.dictproj_check_status(stream()) == 0  # every word is cleared
