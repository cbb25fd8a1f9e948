"""The AdamW step over many tensors: bit for bit the stated fp32 arithmetic, states in 32 and 8 bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import adapter_reference as ref  # noqa: E402
import dictionary_compressed_linear_b200 as dp  # noqa: E402

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05, grad_scale=0.5)
NAMES = ("p", "g", "m", "v", "copy", "m_scale", "v_scale")


def stream():
    return torch.cuda.current_stream().cuda_stream


def host_tensor(n, bits, seed):
    r = np.random.default_rng(seed)
    t = {"p": r.standard_normal(n), "g": r.standard_normal(n) * np.exp(2 * r.standard_normal(n))}
    t["g"][r.random(n) < 0.1] = 0.0
    m, v = r.standard_normal(n) * 0.1, r.random(n) ** 4
    if n > 300:
        m[128:256], v[128:256], t["g"][128:256] = 0, 0, 0  # a block that has never moved
    t = {k: x.astype(np.float32) for k, x in t.items()}
    if bits == 32:
        return {**t, "m": m.astype(np.float32), "v": v.astype(np.float32)}
    blocks = -(-n // 128)
    t["m"] = ref.e4m3_nearest(np.clip(m * 1000, -448, 448))
    t["v"] = ref.e4m3_nearest(np.clip(np.sqrt(v) * 400, 0, 448))
    t["m_scale"], t["v_scale"] = (np.exp(r.standard_normal(blocks) - 7).astype(np.float32) for _ in range(2))
    return t


def on_device(t, shift=0):
    """Device arrays, each starting `shift` elements into its allocation."""
    d = {}
    for k, x in {**t, "copy": np.zeros(t["p"].size, np.float16)}.items():
        whole = torch.zeros(x.size + shift + 1, dtype=torch.from_numpy(x).dtype, device="cuda")
        d[k] = whole[shift:shift + x.size]
        d[k].copy_(torch.from_numpy(x))
    return d


def entry(d, copy=True):
    return {"n": d["p"].numel(), **{k: d[k].data_ptr() for k in NAMES if k in d and (copy or k != "copy")}}


def check(d, want, what):
    for k, x in want.items():
        got = d[k].cpu().numpy()
        same = got.view(np.uint8).tobytes() == np.ascontiguousarray(x).view(np.uint8).tobytes()
        assert same, f"{what}: {k}, first at {np.flatnonzero(got != x)[:3]}"


SIZES = [1, 2, 3, 31, 127, 128, 129, 255, 1000, 2047, 2048, 2049, 4096, 10007, 0, 65536]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_steps_bit_for_bit(bits, shift):
    hosts = [host_tensor(n, bits, 100 + i) for i, n in enumerate(SIZES)]
    devs = [on_device(t, shift) for t in hosts]
    plan = dp.dictproj_adamw_create([entry(d, copy=i % 3 != 1) if d["p"].numel() else {"p": 0, "g": 0, "m": 0, "v": 0, "n": 0}
                                     for i, d in enumerate(devs)], bits)
    for step in (1, 2, 3, 700):
        dp.dictproj_adamw_step(plan, step, stream=stream(), **HYPER)
        hosts = [ref.adamw(t, step, bits=bits, **HYPER) if t["p"].size else t for t in hosts]
    torch.cuda.synchronize()
    for i, (t, d) in enumerate(zip(hosts, devs)):
        if t["p"].size:
            want = dict(t) if i % 3 != 1 else {**t, "copy": np.zeros(t["p"].size, np.float16)}
            check(d, want, f"n={t['p'].size}")


BAD = {"one nan": {5: np.nan}, "a lane of nans": {132: np.nan, 133: np.nan, 134: np.nan, 135: np.nan}, "an infinity": {300: np.inf},
       "minus infinity": {511: -np.inf}, "both": {640: np.inf, 700: np.nan}, "the last": {999: np.nan}, "an infinity in a short block": {990: np.inf},
       "a whole block of nans": {i: np.nan for i in range(256, 384)}}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("what", list(BAD))
def test_a_gradient_that_is_not_finite_spreads_as_stated(what, shift, bits):
    n = 1000
    t = host_tensor(n, bits, 77)
    t["g"][list(BAD[what])] = list(BAD[what].values())
    d = on_device(t, shift)
    plan = dp.dictproj_adamw_create([entry(d)], bits)
    touched = np.zeros(n, bool)
    for i in BAD[what]:
        touched[i if bits == 32 else slice(i // 128 * 128, i // 128 * 128 + 128)] = True
    value = lambda t, k: ref.e4m3_value(t[k]) * ref.each(t[k + "_scale"], n) if bits == 8 else t[k]  # noqa: E731
    for step in (1, 2):  # the second with a clean gradient: what the states carry on
        dp.dictproj_adamw_step(plan, step, stream=stream(), **HYPER)
        with np.errstate(invalid="ignore", over="ignore"):
            t = ref.adamw(t, step, bits=bits, **HYPER)
        torch.cuda.synchronize()
        got = {k: x.cpu().numpy() for k, x in d.items()}
        with np.errstate(invalid="ignore"):
            values = {k: (value(got, k), value(t, k)) for k in ("m", "v")}
        for k, (a, b) in values.items():
            assert np.array_equal(a, b, equal_nan=True), (step, k)
            assert np.array_equal(got[k][~touched], t[k][~touched]), (step, k)  # and what they are held as
            assert not np.isfinite(a[list(BAD[what])]).any()
        for k in ("p", "copy", "m_scale", "v_scale"):
            if k in t:
                assert np.array_equal(got[k], t[k], equal_nan=True), (step, k)
        assert np.isfinite(got["p"][~touched]).all() and np.isfinite(values["m"][0][~touched]).all()
        if bits == 8:
            assert not np.isfinite(values["m"][0][touched]).any()
        clean = host_tensor(n, bits, 78)["g"]
        t["g"] = clean
        d["g"].copy_(torch.from_numpy(clean))


def test_scales_at_the_ends_of_the_fast_quotient():
    # blocks whose scale crosses 2^-90 and 2^100, elements down to the subnormals: bit for bit all the same
    r = np.random.default_rng(11)
    n = 128 * 96
    top = np.concatenate([np.linspace(-93, -87, 48), np.linspace(97, 103, 48)])[:, None]  # of log2 of the block's scale
    size = np.minimum(2.0 ** (top + 8.7 - 45 * r.random((96, 128)) ** 2), 2.0 ** 127)
    size[:, 0] = 2.0 ** (top[:, 0] + 8.7)
    g = (size * r.choice([-1, 1], size.shape) * 10).reshape(-1).astype(np.float32)  # m' = 0.1 g
    t = {"p": r.standard_normal(n).astype(np.float32), "g": g, "m": np.zeros(n, np.uint8), "v": np.zeros(n, np.uint8),
         "m_scale": np.ones(n // 128, np.float32), "v_scale": np.ones(n // 128, np.float32)}
    d = on_device(t)
    plan = dp.dictproj_adamw_create([entry(d)], 8)
    hyper = {**HYPER, "grad_scale": 1.0, "lr": 0.0}
    dp.dictproj_adamw_step(plan, 1, stream=stream(), **hyper)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        t = ref.adamw(t, 1, bits=8, **hyper)
    assert (np.abs(np.log2(t["m_scale"][:48].astype(float)) + 90) < 4).all()
    for k in ("m", "m_scale"):
        assert np.array_equal(d[k].cpu().numpy(), t[k]), k
    low = slice(0, 128 * 48)  # above, v' overflows
    assert np.array_equal(d["v"].cpu().numpy()[low], t["v"][low]) and np.array_equal(d["p"].cpu().numpy()[low], t["p"][low])


def test_what_lies_between_the_tensors_is_not_touched():
    n, total = 130, 400
    arena = {k: torch.full((total,), 5.0, device="cuda") for k in "pgmv"}
    plan = dp.dictproj_adamw_create([{"n": n, **{k: arena[k].data_ptr() + 4 * at for k in "pgmv"}} for at in (0, 201)], 32)
    dp.dictproj_adamw_step(plan, 1, stream=stream(), **HYPER)
    torch.cuda.synchronize()
    for k in "pmv":
        assert (arena[k][n:201] == 5).all() and (arena[k][331:] == 5).all()
        assert (arena[k][:n] != 5).all() and (arena[k][201:331] != 5).all()
    assert (arena["g"] == 5).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_in_one_arena_and_shared_gradients(bits):
    # arrays that touch and gradients that several tensors read are accepted, and every tensor gets its own step
    n, count = 640, 3
    hosts = [host_tensor(n, bits, 40 + i) for i in range(count)]
    arena = {k: torch.from_numpy(np.concatenate([t[k] for t in hosts])).cuda() for k in hosts[0]}
    for t in hosts:
        t["g"] = hosts[0]["g"]
    at = lambda k, i: arena[k].data_ptr() + i * hosts[0][k].nbytes  # noqa: E731
    plan = dp.dictproj_adamw_create([{"n": n, **{k: at(k, 0 if k == "g" else i) for k in arena}} for i in range(count)], bits)
    dp.dictproj_adamw_step(plan, 3, stream=stream(), **HYPER)
    torch.cuda.synchronize()
    want = [ref.adamw(t, 3, bits=bits, **HYPER) for t in hosts]
    for k in arena:
        if k != "g":
            got, exact = arena[k].cpu().numpy(), np.concatenate([w[k] for w in want])
            assert got.tobytes() == exact.tobytes(), k


def test_a_state_in_8_bits_follows_its_32_bit_one():
    # a constant spread of gradients: v tends to g^2. The dithered codes are unbiased, each step adds a
    # rounding of at most 2^-3 of r, forgotten at the rate 1 - beta2; over 4096 elements the mean of
    # r / |g| must come back to 1 within a few per cent where round-to-nearest would never leave its start.
    n, beta2 = 4096, 0.98
    g = torch.exp(torch.linspace(-1, 1, n, device="cuda"))
    t = {"p": torch.zeros(n, device="cuda"), "g": g, "m": torch.zeros(n, dtype=torch.uint8, device="cuda"),
         "v": torch.zeros(n, dtype=torch.uint8, device="cuda"), "m_scale": torch.ones(n // 128, device="cuda"),
         "v_scale": torch.ones(n // 128, device="cuda")}
    plan = dp.dictproj_adamw_create([{"n": n, **{k: x.data_ptr() for k, x in t.items()}}], 8)
    for step in range(1, 401):
        dp.dictproj_adamw_step(plan, step, 0.0, 0.9, beta2, 1e-8, 0.0, 1.0, stream())
    torch.cuda.synchronize()
    r = t["v"].view(torch.float8_e4m3fn).float() * t["v_scale"].repeat_interleave(128)
    m = t["m"].view(torch.float8_e4m3fn).float() * t["m_scale"].repeat_interleave(128)
    assert abs((r / g).mean().item() - 1) < 0.03
    assert ((m / g - 1).abs() <= 0.4).all()  # nearest codes of beta1 = 0.9: stuck within 2^-4 / (1 - beta1)


def test_a_captured_step_and_another_stream():
    t = host_tensor(5000, 8, 9)
    d = on_device(t)
    plan = dp.dictproj_adamw_create([entry(d)], 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dp.dictproj_adamw_step(plan, 5, stream=side.cuda_stream, **HYPER)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dp.dictproj_adamw_step(plan, 6, stream=side.cuda_stream, **HYPER)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for step in (5, 6, 6):
        t = ref.adamw(t, step, bits=8, **HYPER)
    check(d, t, "captured")


@pytest.mark.parametrize("change,status", [(dict(lr=-1.0), -5), (dict(beta1=1.0), -5), (dict(beta2=-0.1), -5),
                                           (dict(eps=-1e-9), -5), (dict(lr=float("nan")), -10),
                                           (dict(grad_scale=float("inf")), -10), (dict(weight_decay=-1.0), -5)])
def test_refused_factors(change, status):
    d = on_device(host_tensor(10, 32, 1))
    before = {k: x.clone() for k, x in d.items()}
    plan = dp.dictproj_adamw_create([entry(d)], 32)
    with pytest.raises(dp.DictprojError) as e:
        dp.dictproj_adamw_step(plan, 1, stream=stream(), **{**HYPER, **change})
    assert e.value.status == status
    with pytest.raises(dp.DictprojError) as e:
        dp.dictproj_adamw_step(plan, 0, stream=stream(), **HYPER)
    assert e.value.status == -5
    torch.cuda.synchronize()
    assert all(torch.equal(d[k], before[k]) for k in d)
