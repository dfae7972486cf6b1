"""Cases of the adapter operators beside a packed projection, each with its plain form.

Four operators, as one layer meets them when adapters are served or trained beside a frozen packed weight:

* ``lora_forward``   Y = base + s (X A^T) U for rows of many requests, each row with its own adapter or none
* ``lora_backward``  dX, dA and dU of it, from X or from the 8-bit checkpoint of X
* ``checkpoint``     X kept in 8 bits for the backward pass and restored
* ``grad_input``     the packed W4A4 layer's input gradient, dX = dY W^

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` makes one pass.
"""

import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one request generates: the text encoder's MLP up projection, one token, one adapter of rank 16
        {"name": "decode one", "op": "lora_forward", "M": 1, "K": 2560, "N": 9728, "rank": 16, "adapters": 1, "mix": "one",
         "save": False},
        # 64 requests generate at once, each with its own choice of 48 adapters in the pool, some with none
        {"name": "decode many", "op": "lora_forward", "M": 64, "K": 2560, "N": 9728, "rank": 16, "adapters": 48,
         "mix": "rows", "save": False},
        # a batch of short prompts, back to back, through the MLP down projection
        {"name": "prompts 130", "op": "lora_forward", "M": 130, "K": 9728, "N": 2560, "rank": 32, "adapters": 3,
         "mix": "runs", "save": False},
        # an image's tokens through an attention projection, one adapter, V kept for the backward pass
        {"name": "image forward", "op": "lora_forward", "M": 4096, "K": 3072, "N": 3072, "rank": 64, "adapters": 1,
         "mix": "one", "save": True},
        # two images of four requests through the MLP up projection, every request its own wide adapter
        {"name": "images of four", "op": "lora_forward", "M": 8192, "K": 3072, "N": 12288, "rank": 128, "adapters": 4,
         "mix": "runs", "save": False},
        # training: a padded batch of several requests' prompts, small layer
        {"name": "backward ragged", "op": "lora_backward", "M": 777, "K": 512, "N": 256, "rank": 8, "adapters": 5,
         "mix": "runs", "kept": "bf16"},
        # training: an attention projection, one adapter, its input kept as it is
        {"name": "backward image", "op": "lora_backward", "M": 4096, "K": 3072, "N": 3072, "rank": 64, "adapters": 1,
         "mix": "one", "kept": "bf16"},
        # training: the MLP down projection, whose wide input is kept in 8 bits
        {"name": "backward kept in 8 bits", "op": "lora_backward", "M": 8192, "K": 12288, "N": 3072, "rank": 32,
         "adapters": 1, "mix": "one", "kept": "int8"},
        # a prompt's activations kept and restored
        {"name": "checkpoint prompt", "op": "checkpoint", "M": 130, "K": 2560},
        # the MLP's hidden activations of two images kept and restored
        {"name": "checkpoint images", "op": "checkpoint", "M": 8192, "K": 12288},
        # the text encoder's MLP down projection, a short prompt's gradient, scales by row
        {"name": "input gradient prompt", "op": "grad_input", "M": 130, "K": 9728, "N": 2560, "group": 256, "by_row": True},
        # the DiT MLP up projection, two images
        {"name": "input gradient images", "op": "grad_input", "M": 8192, "K": 3072, "N": 12288, "group": 256,
         "by_row": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora_forward", "lora_forward", "lora_forward", "lora_backward", "lora_backward", "checkpoint",
                     "grad_input"])
    if op == "checkpoint":
        return {"op": op, "M": _log(rng, 1, 8192), "K": 256 * _log(rng, 1, 48)}
    if op == "grad_input":
        return {"op": op, "M": _log(rng, 1, 4096), "K": 1024 * rng.randint(1, 6), "N": 8 * _log(rng, 16, 1024),
                "group": rng.choice([16, 64, 256, 1024]), "by_row": rng.random() < 0.5}
    mix = rng.choice(["one", "runs", "runs", "rows"])
    M = _log(rng, 1, 256) if mix == "rows" else _log(rng, 1, 6000)
    case = {"op": op, "M": M, "K": 8 * _log(rng, 32, 1280), "N": 8 * _log(rng, 32, 1280),
            "rank": rng.choice([4, 8, 12, 16, 16, 24, 32, 32, 64, 64, 100, 128]),
            "adapters": 1 if mix == "one" else _log(rng, 2, 24), "mix": mix}
    if op == "lora_forward":
        case["save"] = rng.random() < 0.4
    else:
        case["kept"] = rng.choice(["bf16", "int8"])
        if case["kept"] == "int8":
            case["K"] = 256 * _log(rng, 1, 40)
    return case


# ---------------------------------------------------------------------------------------------- inputs

def _bf(g, *shape, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(BF16)


def _activations(g, M, K):
    """Normal values with 1 % of the channels 50 times as large, as the layer's inputs have them."""
    x = torch.randn(M, K, device="cuda", generator=g)
    loud = torch.rand(K, device="cuda", generator=g) < 0.01
    return torch.where(loud, x * 50, x).to(BF16)


def _rows_adapters(case, g):
    """The adapter of each row, int32 [M], -1 for none; None where every row has the pool's only adapter."""
    M, L = case["M"], case["adapters"]
    if case["mix"] == "one":
        return None
    if case["mix"] == "rows":  # each row its own, one in eight with none
        a = torch.randint(0, L, (M,), device="cuda", generator=g, dtype=torch.int32)
        return torch.where(torch.rand(M, device="cuda", generator=g) < 0.125, torch.full_like(a, -1), a)
    # runs of rows: L + 1 borders drawn over the rows; the rows behind the last are padding
    cuts = torch.sort(torch.rand(L - 1, device="cuda", generator=g)).values * M
    end = M - max(0, min(M // 50, 64))
    pos = torch.arange(M, device="cuda")
    a = torch.searchsorted(cuts, pos.float(), right=True)
    order = torch.randperm(L, device="cuda", generator=g)
    return torch.where(pos < end, order[a], torch.full_like(pos, -1)).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    if op == "checkpoint":
        return {"case": case, "X": _activations(g, M, K)}
    N = case["N"]
    if op == "grad_input":
        codes = torch.clamp(torch.round(torch.randn(N, K, device="cuda", generator=g) * 1.7), -7, 7).to(torch.int32)
        packed = ((codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)).to(torch.uint8)
        s = 0.01 + 0.005 * torch.rand(N if case["by_row"] else 1, device="cuda", generator=g)
        return {"case": case, "dY": _bf(g, M, N, std=1e-3), "Wq": packed, "w_scale": s.expand(N).contiguous()}
    L, r = case["adapters"], case["rank"]
    s = {"case": case, "X": _activations(g, M, K), "down": _bf(g, L, r, K, std=K ** -0.5),
         "up": _bf(g, L, r, N, std=0.02), "scale": 16.0 / r * (0.5 + torch.rand(L, device="cuda", generator=g)),
         "adapter": _rows_adapters(case, g)}
    if op == "lora_forward":
        s["base"] = _bf(g, M, N)
        return s
    s["V"] = _lora_v(s["X"].float(), s["down"].float(), s["adapter"]).to(BF16)
    s["dY"] = _bf(g, M, N, std=1e-3)
    s["base"] = _bf(g, M, K, std=1e-3)
    if case["kept"] == "int8":
        s["codes"], s["code_scales"] = _codes(s.pop("X").float())
    return s


# ---------------------------------------------------------------------------------------------- plain forms

def _hadamard(group, dtype, device):
    """H_group: Kronecker power of J - 2I of order 4, over sqrt(group); symmetric, its own inverse."""
    h4 = torch.ones(4, 4, dtype=dtype, device=device) - 2 * torch.eye(4, dtype=dtype, device=device)
    h16 = torch.kron(h4, h4)
    h = {16: h16, 64: torch.kron(h16, h4), 256: torch.kron(h16, h16)}.get(group)
    h = torch.kron(torch.kron(h16, h16), h4) if h is None else h
    return h / group ** 0.5


def _rotate(x, group=256):
    return (x.reshape(x.shape[0], -1, group) @ _hadamard(group, x.dtype, x.device)).reshape(x.shape)


def _codes(x):
    """8-bit codes of the rotated rows, and one float32 scale for each row and 256 columns."""
    y = _rotate(x).reshape(x.shape[0], -1, 256)
    s = (y.abs().amax(-1) / 127).float()
    s = torch.where(s > 0, s, torch.ones_like(s))
    return torch.round(y / s.to(y.dtype)[..., None]).to(torch.int8).reshape(x.shape), s


def _values(codes, scales, dtype):
    """What the codes stand for: codes times scale, rotated back."""
    c = codes.to(dtype).reshape(codes.shape[0], -1, 256) * scales.to(dtype)[..., None]
    return _rotate(c.reshape(codes.shape))


def _spread(v, adapter, L):
    """[M, r] -> [M, L r]: each row's values in its adapter's columns, zeros in the others'."""
    if adapter is None:
        return v
    mine = adapter.long()[:, None] == torch.arange(L, device=v.device)
    return (v[:, None, :] * mine[..., None].to(v.dtype)).reshape(v.shape[0], -1)


def _own_columns(v, adapter, L):
    """[M, L r] -> [M, r]: each row's own adapter's columns, zeros where it has none."""
    if adapter is None:
        return v
    a = adapter.long()
    v = v.reshape(v.shape[0], L, -1)
    v = v[torch.arange(v.shape[0], device=v.device), a.clamp(0, L - 1)]
    return torch.where(((a >= 0) & (a < L))[:, None], v, torch.zeros_like(v))


def _row_scale(scale, adapter):
    return scale[0] if adapter is None else scale[adapter.long().clamp(0, scale.shape[0] - 1)][:, None]


def _lora_v(x, down, adapter):
    L, r, K = down.shape
    return _own_columns(x @ down.reshape(L * r, K).T, adapter, L)


def _plain_forward(s, dtype):
    down, up, a = s["down"].to(dtype), s["up"].to(dtype), s["adapter"]
    L, r, N = up.shape
    v = _lora_v(s["X"].to(dtype), down, a)
    y = s["base"].to(dtype) + _spread(v * _row_scale(s["scale"].to(dtype), a), a, L) @ up.reshape(L * r, N)
    return {"Y": y, "V": v} if s["case"]["save"] else {"Y": y}


def _plain_backward(s, dtype):
    down, up, a, dy = s["down"].to(dtype), s["up"].to(dtype), s["adapter"], s["dY"].to(dtype)
    L, r, K = down.shape
    N = up.shape[2]
    x = s["X"].to(dtype) if "X" in s else _values(s["codes"], s["code_scales"], dtype)
    sc = _row_scale(s["scale"].to(dtype), a)
    dv = _spread(sc * _own_columns(dy @ up.reshape(L * r, N).T, a, L), a, L)
    dx = s["base"].to(dtype) + dv @ down.reshape(L * r, K)
    du = _spread(sc * s["V"].to(dtype), a, L).T @ dy
    return {"dX": dx, "d_down": (dv.T @ x).reshape(L, r, K), "d_up": du.reshape(L, r, N)}


def _plain_checkpoint(s, dtype):
    return {"X": _values(*_codes(s["X"].to(dtype)), dtype)}


def _plain_grad_input(s, dtype):
    w = s["Wq"].to(torch.int32)
    q = torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], -1)
    q = torch.where(q > 7, q - 16, q).to(dtype) * s["w_scale"].to(dtype)[:, None]
    return {"dX": s["dY"].to(dtype) @ _rotate(q, s["case"]["group"])}


PLAIN = {"lora_forward": _plain_forward, "lora_backward": _plain_backward, "checkpoint": _plain_checkpoint,
         "grad_input": _plain_grad_input}


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {k: v.to(BF16) for k, v in PLAIN[op](s, torch.float32).items()}
    import w4a8_rotated_quantized_b200 as cr

    if op == "lora_forward":
        out = cr.cr_lora_forward(s["X"], s["down"], s["up"], s["scale"], adapter=s["adapter"], base=s["base"],
                                 save_v=s["case"]["save"])
        return {"Y": out[0], "V": out[1]} if s["case"]["save"] else {"Y": out}
    if op == "lora_backward":
        kept = s["X"] if "X" in s else (s["codes"], s["code_scales"])
        dx, dd, du = cr.cr_lora_backward(s["dY"], kept, s["V"], s["down"], s["up"], s["scale"], adapter=s["adapter"],
                                         base=s["base"])
        return {"dX": dx, "d_down": dd, "d_up": du}
    if op == "checkpoint":
        return {"X": cr.cr_ckpt_load(*cr.cr_ckpt_save(s["X"]))}
    return {"dX": cr.cr_w4a4_grad_input(s["dY"], s["Wq"], s["w_scale"], group=s["case"]["group"])}


# ---------------------------------------------------------------------------------------------- 64 bits

def _h64(group):
    """Entry (i, j) of H_group from the index bits: -1 for each base-4 digit that agrees, over sqrt(group)."""
    i = torch.arange(group, device="cuda")
    h = torch.ones(group, group, dtype=torch.float64, device="cuda")
    d = 1
    while d < group:
        h = h * torch.where(((i // d) % 4)[:, None] == ((i // d) % 4)[None, :], -1.0, 1.0)
        d *= 4
    return h / math.sqrt(group)


def _each(adapter, M, L):
    """(adapter, its rows) for every adapter of the pool."""
    rows = torch.arange(M, device="cuda")
    return [(l, rows if adapter is None else torch.nonzero(adapter == l)[:, 0]) for l in range(L)]


def exact(case, seed):
    s = prepare(case, seed)
    f = lambda k: s[k].double()  # noqa: E731
    op, M, K = case["op"], case["M"], case["K"]
    if op == "grad_input":
        lo, hi = s["Wq"] % 16, s["Wq"] // 16
        q = torch.empty(case["N"], K, dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = lo.double() - 16 * (lo > 7), hi.double() - 16 * (hi > 7)
        h, n = _h64(case["group"]), case["group"]
        dz = (f("dY") * f("w_scale")) @ q
        return {"dX": torch.einsum("mgi,ij->mgj", dz.view(M, K // n, n), h).reshape(M, K)}
    if op == "checkpoint":
        h, out = _h64(256), []
        for x in f("X").split(1024):
            y = x.view(-1, 256) @ h
            sc = (y.abs().max(1).values / 127).float().double()
            sc[sc == 0] = 1
            out.append(((torch.round(y / sc[:, None]) * sc[:, None]) @ h).view(-1, K))
        return {"X": torch.cat(out)}
    L, r, N = case["adapters"], case["rank"], case["N"]
    if op == "lora_forward":
        y, v = f("base"), torch.zeros(M, r, dtype=torch.float64, device="cuda")
        for l, rows in _each(s["adapter"], M, L):
            v[rows] = f("X")[rows] @ s["down"][l].double().T
            y[rows] += s["scale"][l].double() * (v[rows] @ s["up"][l].double())
        return {"Y": y, "V": v} if case["save"] else {"Y": y}
    if case["kept"] == "int8":
        c = s["codes"].double().view(M, K // 256, 256) * f("code_scales")[:, :, None]
        x = (c.view(-1, 256) @ _h64(256)).view(M, K)
    else:
        x = f("X")
    dx, dy = f("base"), f("dY")
    dd = torch.zeros(L, r, K, dtype=torch.float64, device="cuda")
    du = torch.zeros(L, r, N, dtype=torch.float64, device="cuda")
    for l, rows in _each(s["adapter"], M, L):
        sc = s["scale"][l].double()
        dv = sc * (dy[rows] @ s["up"][l].double().T)
        dx[rows] += dv @ s["down"][l].double()
        dd[l] = dv.T @ x[rows]
        du[l] = sc * (s["V"][rows].double().T @ dy[rows])
    return {"dX": dx, "d_down": dd, "d_up": du}


# ---------------------------------------------------------------------------------------------- work

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "checkpoint":  # X in, codes and scales out and in again, X out
        return {"bytes": 2 * M * K * 2 + 2 * M * (K + K // 64), "flops": 2 * 2 * M * K * 16}
    N = case["N"]
    if op == "grad_input":
        return {"bytes": 2 * M * (N + K) + N * K // 2 + 4 * N, "flops": 2 * M * N * K}
    L, r = case["adapters"], case["rank"]
    used = min(L, M) if case["mix"] != "one" else 1
    pool = 2 * used * r * (K + N)
    if op == "lora_forward":
        return {"bytes": 2 * M * (K + 2 * N) + pool + (2 * M * r if case["save"] else 0), "flops": 2 * M * r * (K + N)}
    kept = M * (K + K // 64) if case["kept"] == "int8" else 2 * M * K
    return {"bytes": 2 * M * (N + 2 * K + r) + kept + pool + 2 * L * r * (K + N), "flops": 4 * M * r * (K + N)}
