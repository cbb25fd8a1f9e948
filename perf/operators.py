"""Measured cases of the operators that train and serve low-rank adapters on compressed projections.

The operators: the adapters' forward over the rows of many requests, their backward pass, the input gradient of the
frozen projection Y = X D C, and the AdamW step over many tensors with states in 32 or 8 bits. `run` computes each in
elementary torch operations, or, where `own` is set, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

HALF = torch.float16
BLOCK = 128  # elements that share the scale of an 8-bit state
TINY = 2.0 ** -126  # the smallest scale


# ---------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one request in a decode step, an attention projection
        {"name": "forward 1 row", "op": "forward", "rows": 1, "slots": 8, "used": 1, "none": 0, "rank": 16, "ragged": False, "d_in": 4096, "d_out": 4096},
        # a decode step of 64 requests, each with an adapter of its own, the widest projection
        {"name": "forward 64 requests", "op": "forward", "rows": 64, "slots": 64, "used": 64, "none": 0, "rank": 16, "ragged": False, "d_in": 4096, "d_out": 11008},
        # an odd batch: odd widths, adapters of several ranks, rows of requests without an adapter
        {"name": "forward ragged", "op": "forward", "rows": 37, "slots": 6, "used": 5, "none": 9, "rank": 24, "ragged": True, "d_in": 1376, "d_out": 1001},
        # prompts of four requests in one prefill call
        {"name": "forward 2048 rows", "op": "forward", "rows": 2048, "slots": 8, "used": 4, "none": 0, "rank": 32, "ragged": False, "d_in": 4096, "d_out": 4096},
        # a short training sequence on a small layer of odd width, three adapters trained at once
        {"name": "backward ragged", "op": "backward", "rows": 100, "slots": 4, "used": 3, "none": 7, "rank": 12, "ragged": True, "d_in": 1376, "d_out": 1001},
        # one adapter, one training sequence, the widest projection
        {"name": "backward 2048 rows", "op": "backward", "rows": 2048, "slots": 1, "used": 1, "none": 0, "rank": 16, "ragged": False, "d_in": 4096, "d_out": 11008},
        # the largest micro-batch, adapters of a high rank
        {"name": "backward 8192 rows", "op": "backward", "rows": 8192, "slots": 3, "used": 3, "none": 0, "rank": 64, "ragged": False, "d_in": 4096, "d_out": 4096},
        # the input gradient of one short sequence through an attention projection
        {"name": "input gradient 128 rows", "op": "input", "rows": 128, "d_in": 4096, "k": 2048, "d_out": 4096, "density": 0.3},
        # the input gradient of a full sequence through the widest projection
        {"name": "input gradient 2048 rows", "op": "input", "rows": 2048, "d_in": 4096, "k": 2048, "d_out": 11008, "density": 0.3},
        # the adapters of one layer, states in 32 bits
        {"name": "adamw 32 one layer", "op": "adamw", "bits": 32, "tensors": 14, "mean": 65536, "ragged": False},
        # the adapters of a whole stack of 224 projections, states in 8 bits
        {"name": "adamw 8 whole stack", "op": "adamw", "bits": 8, "tensors": 448, "mean": 98304, "ragged": False},
        # tensors of odd sizes, some shorter than a block of the states
        {"name": "adamw 8 ragged", "op": "adamw", "bits": 8, "tensors": 61, "mean": 20011, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "input", "adamw", "adamw"])
    if op in ("forward", "backward"):
        rows = _log(rng, 1, 8192 if op == "backward" else 4096)
        rank = _log(rng, 1, 128)
        slots = min(_log(rng, 1, 64), max(1, 2048 // rank))
        used = rng.randint(1, min(slots, rows))
        none = rng.choice([0, 0, rng.randint(0, max(0, rows - used) // 4)])
        d_in = 32 * _log(rng, 4, 344 if rows <= 2048 else 128)
        d_out = rng.choice([8, 8, 1]) * _log(rng, 8, 1376 if rows <= 2048 else 512)
        return {"op": op, "rows": rows, "slots": slots, "used": used, "none": none, "rank": rank,
                "ragged": rng.random() < 0.5, "d_in": d_in, "d_out": d_out}
    if op == "input":
        return {"op": op, "rows": _log(rng, 1, 2048), "d_in": 32 * _log(rng, 4, 128), "k": 16 * _log(rng, 4, 128),
                "d_out": 8 * _log(rng, 8, 1376), "density": round(rng.uniform(0.2, 0.4), 3)}
    tensors = _log(rng, 1, 448)
    bits = rng.choice([8, 32])
    return {"op": op, "bits": bits, "tensors": tensors, "mean": _log(rng, 100, min(4 << 20, (44 if bits == 8 else 26) * (1 << 20) // tensors)),
            "ragged": rng.random() < 0.7}


def _counts(case):
    """Rows of each used slot: the first has the most, every one at least one."""
    left = case["rows"] - case["none"] - case["used"]
    w = [1.0 / (1 + i) for i in range(case["used"])]
    c = [1 + int(left * x / sum(w)) for x in w]
    c[0] += case["rows"] - case["none"] - sum(c)
    return c


def _ranks(case):
    r = case["rank"]
    return [r if not case["ragged"] else max(1, r - (5 * s) % r) for s in range(case["slots"])]


def _sizes(case):
    """Elements of each tensor."""
    n, mean = case["tensors"], case["mean"]
    if not case["ragged"]:
        return [mean] * n
    return [max(1, (mean * (1 + 37 * i % 97)) // 49 + i % 3) for i in range(n)]


def work(case):
    if case["op"] in ("forward", "backward"):
        counts, ranks = _counts(case), _ranks(case)
        i, o, rows = case["d_in"], case["d_out"], case["rows"]
        used = sum(ranks[: case["used"]])
        mac = sum(c * r for c, r in zip(counts, ranks))
        if case["op"] == "forward":
            return {"bytes": 2 * (rows - case["none"]) * i + 4 * rows * o + 2 * used * (i + o), "flops": 2 * mac * (i + o)}
        grads = 4 * case["slots"] * case["rank"] * (i + o)
        return {"bytes": 2 * (rows - case["none"]) * (i + o) + 4 * rows * i + 2 * used * (i + o) + grads, "flops": 6 * mac * (i + o)}
    if case["op"] == "input":
        m, i, k, o = case["rows"], case["d_in"], case["k"], case["d_out"]
        kept = math.ceil(case["density"] * k)
        packed = i * k * 9 / 16 + o * kept * 25 / 16
        return {"bytes": 2 * m * (i + o) + packed, "flops": 2 * m * (k * i + kept * o)}
    n = sum(_sizes(case))
    # p read and written, g read, the fp16 copy written, two states read and written
    return {"bytes": n * (14 + (16 if case["bits"] == 32 else 4)) + (0 if case["bits"] == 32 else 16 * (n // BLOCK)), "flops": 16 * n}


# ---------------------------------------------------------------------------------------------- inputs
def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale)

    return g, normal


def _adapter_inputs(case, seed):
    g, normal = _rand(seed)
    i, o, rows, slots, rank = case["d_in"], case["d_out"], case["rows"], case["slots"], case["rank"]
    counts, ranks = _counts(case), _ranks(case)
    runs = [np.full(c, s) for s, c in enumerate(counts)] + [np.full(case["none"], -1)]
    order = np.random.RandomState(seed % (1 << 31)).permutation
    # whole sequences lie one behind the other; the single tokens of a decode step in any order
    ids = np.concatenate([runs[j] for j in order(len(runs))]) if rows >= 256 else order(np.concatenate(runs))
    live = torch.arange(rank, device="cuda")[None, :, None] < torch.tensor(ranks, device="cuda")[:, None, None]
    s = {
        "ids": torch.tensor(ids, dtype=torch.int32, device="cuda"),
        "ranks": ranks,
        "scale": torch.tensor([16.0 / r for r in ranks], device="cuda"),
        "A": (normal(slots, rank, i, scale=i ** -0.5) * live).to(HALF),
        "B": (normal(slots, rank, o, scale=0.02) * live).to(HALF),
    }
    X = normal(rows, i)
    X[:, torch.randperm(i, generator=g, device="cuda")[: round(0.01 * i)]] *= 20.0  # outlier channels
    s["X"] = X.to(HALF)
    if case["op"] == "forward":
        s["base"] = normal(rows, o).to(HALF)  # the shared projection's result
    else:
        s["dY"] = normal(rows, o, scale=0.02).to(HALF)
        s["base"] = normal(rows, i, scale=0.02).to(HALF)  # the input gradient of the shared projection
    return s


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes(x):
    """4-bit codes of values near to the grid's range, and what they stand for."""
    grid = torch.tensor(E2M1, device="cuda")
    mag = torch.bucketize(x.abs(), (grid[1:] + grid[:-1]) / 2)
    code = torch.where((x < 0) & (mag > 0), mag + 8, mag).to(torch.uint8)
    return code, torch.where(x < 0, -grid[mag], grid[mag])


def _scales(shape, g):
    """E4M3 scale codes of the upper range, and what they stand for."""
    c = torch.randint(0x68, 0x7F, shape, generator=g, device="cuda").to(torch.uint8)
    return c, c.view(torch.float8_e4m3fn).float()


def _projection_inputs(case, seed):
    """A packed dictionary and coefficient matrix (codes, scales, support) and their dense values."""
    g, normal = _rand(seed)
    i, k, o = case["d_in"], case["k"], case["d_out"]
    dc, dv = _codes(normal(k, i, scale=2.0))
    ds, dsv = _scales((k, i // 16), g)
    s_d = float(np.float32(1.0 / (400.0 * math.sqrt(i))))
    nnz = math.ceil(case["density"] * k)
    pad = -(-nnz // 16) * 16
    atoms = torch.rand(o, k, generator=g, device="cuda").argsort(dim=1)[:, :nnz].sort(dim=1).values
    cc, cv = _codes(normal(o, nnz, scale=2.0))
    cs, csv = _scales((o, pad // 16), g)
    s_c = float(np.float32(1.0 / (400.0 * math.sqrt(k))))
    cv = cv * csv.repeat_interleave(16, dim=1)[:, :nnz]
    packed = {"dc": dc, "ds": ds, "cc": cc, "cs": cs, "atoms": atoms, "pad": pad, "s_d": s_d, "s_c": s_c}
    D = dv * dsv.repeat_interleave(16, dim=1)  # [k][d_in], without s_d
    C = torch.zeros(o, k, device="cuda").scatter_(1, atoms, cv)  # [d_out][k], without s_c
    return packed, D, C


def _handles(case, p):
    import dictionary_compressed_linear_b200 as dp

    i, k, o, pad = case["d_in"], case["k"], case["d_out"], p["pad"]
    nnz = p["atoms"].shape[1]
    grow = lambda t: torch.nn.functional.pad(t, (0, pad - nnz))  # noqa: E731
    pairs = lambda t: (t[..., 0::2] | (t[..., 1::2] << 4)).flatten().cpu().numpy()  # noqa: E731
    group = dp.dictproj_group_upload({"codes": pairs(p["dc"]), "scales": p["ds"].flatten().cpu().numpy(), "s": p["s_d"], "d_in": i, "k": k}, case["rows"])
    nseg = -(-k // 256)
    starts = torch.searchsorted(p["atoms"].contiguous(), (torch.arange(nseg, device="cuda") * 256).expand(o, nseg).contiguous())
    layer = dp.dictproj_layer_upload({
        "col_ptr": (np.arange(o + 1, dtype=np.int64) * pad).astype(np.uint32), "codes": pairs(grow(p["cc"])),
        "scales": p["cs"].flatten().cpu().numpy(), "idx": grow(p["atoms"] & 255).to(torch.uint8).flatten().cpu().numpy(),
        "seg_start": starts.flatten().cpu().numpy().astype(np.uint16), "s": p["s_c"], "k": k, "d_out": o})
    dp.dictproj_group_reserve_backward(group, o)
    return group, layer


def _adamw_inputs(case, seed):
    """Tensors in one arena, each from a multiple of 128 on."""
    g, normal = _rand(seed)
    sizes = _sizes(case)
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    at = np.concatenate([[0], np.cumsum(room)])
    total = int(at[-1])
    first = torch.tensor(at[:-1], device="cuda")
    index = torch.arange(total, device="cuda") - first.repeat_interleave(torch.tensor(room, device="cuda"))
    live = index < torch.tensor(sizes, device="cuda").repeat_interleave(torch.tensor(room, device="cuda"))
    spread = torch.exp(normal(total // BLOCK)).repeat_interleave(BLOCK)  # gradients of rows differ in size
    s = {"sizes": sizes, "at": at[:-1].tolist(), "index": index, "t": 100 + seed % 7,
         "p": normal(total, scale=0.02) * live, "g": normal(total, scale=1e-3) * spread * live,
         "copy": torch.zeros(total, dtype=HALF, device="cuda")}
    m = normal(total, scale=3e-4) * spread * live
    v = (normal(total, scale=1e-3) * spread).square() * live + m.square()
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["m_scale"] = _encode(m)
        s["v"], s["v_scale"] = _encode(v.sqrt())
    return s


def _block_scale(x):
    return (x.abs().amax(dim=1, keepdim=True) / 448.0).clamp_min(TINY)


def _encode(x):
    x = x.view(-1, BLOCK)
    s = _block_scale(x)
    return (x / s).to(torch.float8_e4m3fn).view(-1).view(torch.uint8), s.view(-1).clone()


LR, BETA1, BETA2, EPS, DECAY, GRAD_SCALE = 2e-4, 0.9, 0.999, 1e-8, 0.01, 0.5


def prepare(case, seed):
    op = case["op"]
    if op in ("forward", "backward"):
        s = _adapter_inputs(case, seed)
    elif op == "input":
        packed, D, C = _projection_inputs(case, seed)
        _, normal = _rand(seed + 1)
        s = {"dY": normal(case["rows"], case["d_out"], scale=0.02).to(HALF)}
        if own:
            s["group"], s["layer"] = _handles(case, packed)
            s["dX"] = torch.empty(case["rows"], case["d_in"], dtype=HALF, device="cuda")
        else:
            s["D"], s["C"] = D * packed["s_d"], C * packed["s_c"]
    else:
        s = _adamw_inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(s, case)
    return s


def _prepare_own(s, case):
    """The handles that a program keeps: the pool of adapters, the plan of the batch's rows, the optimiser's plan."""
    import dictionary_compressed_linear_b200 as dp

    stream = torch.cuda.current_stream().cuda_stream
    rows, slots, rank = case.get("rows"), case.get("slots"), case.get("rank")
    if case["op"] in ("forward", "backward"):
        s["pool"] = dp.dictproj_adapters_create(case["d_in"], case["d_out"], rank, slots, rows)
        for i, r in enumerate(s["ranks"]):
            dp.dictproj_adapters_set(s["pool"], i, r, float(s["scale"][i]), s["A"][i].data_ptr(), s["B"][i].data_ptr(), stream)
        s["rows"] = dp.dictproj_rows_create(rows, slots)
        dp.dictproj_rows_set(s["rows"], s["ids"].data_ptr(), rows, stream)
        s["out"] = torch.empty_like(s["base"])
        if case["op"] == "backward":
            s["dA"] = torch.empty(slots, rank, case["d_in"], device="cuda")
            s["dB"] = torch.empty(slots, rank, case["d_out"], device="cuda")
    elif case["op"] == "adamw":
        eight = case["bits"] == 8
        here = lambda name, at: s[name].data_ptr() + at * s[name].element_size()  # noqa: E731
        s["plan"] = dp.dictproj_adamw_create([
            {"p": here("p", a), "g": here("g", a), "m": here("m", a), "v": here("v", a), "copy": here("copy", a), "n": n,
             "m_scale": here("m_scale", a // BLOCK) if eight else 0, "v_scale": here("v_scale", a // BLOCK) if eight else 0}
            for a, n in zip(s["at"], s["sizes"])], state_bits=case["bits"])


# ---------------------------------------------------------------------------------------------- one pass
def run(s):
    return {"forward": _forward, "backward": _backward, "input": _input, "adamw": _adamw}[s["case"]["op"]](s)


def _spread(s):
    """[rows][slots] scale of the row's own slot, 0 elsewhere."""
    return (s["ids"][:, None] == torch.arange(s["A"].shape[0], device="cuda")) * s["scale"]


def _through(x, weights, spread):
    """x times each slot's weights, of which a row keeps its own slot's: [rows][slots * rank]."""
    slots, rank, _ = weights.shape
    t = x @ weights.flatten(0, 1).T
    return (t.view(-1, slots, rank) * spread[:, :, None]).view(-1, slots * rank)


def _forward(s):
    if own:
        import dictionary_compressed_linear_b200 as dp
        dp.dictproj_adapter_forward(s["pool"], s["rows"], s["X"].data_ptr(), s["base"].data_ptr(), s["out"].data_ptr(),
                                    torch.cuda.current_stream().cuda_stream)
        return s["out"]
    T = _through(s["X"].float(), s["A"].float(), _spread(s))
    return (s["base"].float() + T @ s["B"].float().flatten(0, 1)).to(HALF)


def _backward(s):
    if own:
        import dictionary_compressed_linear_b200 as dp
        dp.dictproj_adapter_backward(s["pool"], s["rows"], s["X"].data_ptr(), s["dY"].data_ptr(), s["base"].data_ptr(), s["out"].data_ptr(),
                                     s["dA"].data_ptr(), s["dB"].data_ptr(), False, torch.cuda.current_stream().cuda_stream)
        return {"dX": s["out"], "dA": s["dA"], "dB": s["dB"]}
    spread, X, dY, A, B = _spread(s), s["X"].float(), s["dY"].float(), s["A"].float(), s["B"].float()
    U, T = _through(dY, B, spread), _through(X, A, spread)
    return {"dX": (s["base"].float() + U @ A.flatten(0, 1)).to(HALF), "dA": (U.T @ X).view(A.shape), "dB": (T.T @ dY).view(B.shape)}


def _input(s):
    if own:
        import dictionary_compressed_linear_b200 as dp
        dp.dictproj_backward_input(s["dY"].data_ptr(), s["dY"].shape[0], s["layer"], s["group"], s["dX"].data_ptr(),
                                   torch.cuda.current_stream().cuda_stream)
        return s["dX"]
    return ((s["dY"].float() @ s["C"]) @ s["D"]).to(HALF)


def _dither(index, t):
    """20 bits from an element's number and the step's: what decides how the second state is rounded."""
    h = (index * 0x9E3779B9 + t * 0x6A09E667) & 0xFFFFFFFF
    h = ((h ^ (h >> 16)) * 0xBB67AE85) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0x6A09E667) & 0xFFFFFFFF
    return h >> 12


def _adamw(s):
    s["t"] += 1
    t, eight = s["t"], s["case"]["bits"] == 8
    names = ("p", "copy", "m", "v") + (("m_scale", "v_scale") if eight else ())
    if own:
        import dictionary_compressed_linear_b200 as dp
        dp.dictproj_adamw_step(s["plan"], t, LR, BETA1, BETA2, EPS, DECAY, GRAD_SCALE, torch.cuda.current_stream().cuda_stream)
    else:
        f = lambda x: float(np.float32(x))  # noqa: E731
        m, v = s["m"], s["v"]
        if eight:
            m = (m.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
            r = (v.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1)
            v = r * r
        g = s["g"] * f(GRAD_SCALE)
        m = m * f(BETA1) + g * f(1.0 - BETA1)
        v = v * f(BETA2) + (g * f(1.0 - BETA2)) * g
        r = v.sqrt()
        step = m / (r * f(1.0 / math.sqrt(1.0 - BETA2 ** t)) + f(EPS))
        s["p"] = s["p"] * f(1.0 - LR * DECAY) - step * f(LR / (1.0 - BETA1 ** t))
        s["copy"] = s["p"].to(HALF)
        if eight:
            s["m"], s["m_scale"] = _encode(m)
            r = r.view(-1, BLOCK)
            scale = _block_scale(r)
            up = _dither(s["index"], t).to(torch.int32)
            code = ((((r / scale) * 2.0 ** -120).view(-1).view(torch.int32) + up) >> 20).clamp_max(0x7E)
            s["v"] = torch.where(r.view(-1) > 0, code.clamp_min(1), code).to(torch.uint8)
            s["v_scale"] = scale.view(-1)
        else:
            s["m"], s["v"] = m, v
    # what 8 bits hold is returned as numbers of its format, beside the scales that they are multiplied with
    return {n: s[n].view(torch.float8_e4m3fn) if eight and n in ("m", "v") else s[n] for n in names}


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "input":
        packed, D, C = _projection_inputs(case, seed)
        _, normal = _rand(seed + 1)
        dY = normal(case["rows"], case["d_out"], scale=0.02).to(HALF).double()
        return torch.linalg.multi_dot([dY, C.double() * packed["s_c"], D.double() * packed["s_d"]])
    if op == "adamw":
        s = _adamw_inputs(case, seed)
        eight = case["bits"] == 8
        t, g = s["t"] + 1, s["g"].double() * GRAD_SCALE
        value = lambda n: s[n].view(torch.float8_e4m3fn).double() * s[n + "_scale"].double().repeat_interleave(BLOCK)  # noqa: E731
        m = BETA1 * (value("m") if eight else s["m"].double()) + (1 - BETA1) * g
        v = BETA2 * (value("v").square() if eight else s["v"].double()) + (1 - BETA2) * g.square()
        hat_m, hat_v = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        p = s["p"].double()
        p = p - LR * (hat_m / (hat_v.sqrt() + EPS) + DECAY * p)
        # a state in 8 bits is a choice between codes: it has no value in 64 bits
        return {"p": p, "copy": p, **({n: None for n in ("m", "v", "m_scale", "v_scale")} if eight else {"m": m, "v": v})}
    s = _adapter_inputs(case, seed)
    ids = s["ids"].cpu().numpy()
    X, A, B = s["X"].double(), s["A"].double(), s["B"].double()
    out = s["base"].double()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for slot, r in enumerate(s["ranks"]):
        at = torch.tensor(np.flatnonzero(ids == slot), device="cuda")
        a, b, w = A[slot, :r], B[slot, :r], 16.0 / r
        if op == "forward":
            out[at] += w * torch.einsum("mi,ri,ro->mo", X[at], a, b)
        else:
            dY = s["dY"][at].double()
            u = w * torch.einsum("mo,ro->mr", dY, b)
            out[at] += torch.einsum("mr,ri->mi", u, a)
            dA[slot, :r] = torch.einsum("mr,mi->ri", u, X[at])
            dB[slot, :r] = w * torch.einsum("mi,ri,mo->ro", X[at], a, dY)
    return out if op == "forward" else {"dX": out, "dA": dA, "dB": dB}
