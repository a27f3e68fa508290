"""Cases of the multi-adapter and 8-bit checkpoint operators, with their plain forms.

Five operators around one frozen NF4 weight W [N, K] and a pool of n low-rank
adapters A [n, r, K], B [n, N, r] with scales s [n]; row m of a batch uses the
adapter index[m], or none where index[m] is outside 0 .. n - 1:

  fwd    y = x . W'^T + s_a (x . A_a^T) . B_a^T                      (a = index[m], row by row)
  bwd    dX = dY . W' + s_a (dY . B_a) . A_a
  grad   dA_a = s_a sum_m (dY . B_a)_m^T x_m,  dB_a = s_a sum_m dY_m^T (x . A_a^T)_m   over the rows of a
  ckpt   an activation kept in 8 bits (blocks of 64 with one bf16 absmax) and restored
  cgrad  dA, dB of one adapter from a layer input that is kept in 8 bits

W' is the bf16 value of the stored NF4 weight: bf16(L[code] * fp32(q * d)).
"""
import torch

own = False

BLOCK, GROUP = 64, 256


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    def case(name, op, M, N, K, r, n=1, requests=1, fmt="int8"):
        return {"name": name, "op": op, "M": M, "N": N, "K": K, "r": r, "n": n, "requests": requests, "fmt": fmt}

    return [
        # one token of one request at an attention projection: the smallest serving call
        case("fwd_1_token", "fwd", 1, 4096, 4096, 16, n=8),
        # a decode step of 48 requests, each with an adapter of its own, at the up projection
        case("fwd_48_requests", "fwd", 48, 11008, 4096, 16, n=64, requests=48),
        # a prefill batch of a few prompts of uneven length, ragged in the end
        case("fwd_prefill_700", "fwd", 700, 4096, 11008, 8, n=16, requests=5),
        # a training batch in which eight adapters train side by side
        case("fwd_train_4096", "fwd", 4096, 11008, 4096, 16, n=8, requests=11),
        # its backward to the input, and that of a short ragged batch at rank 64
        case("bwd_train_4096", "bwd", 4096, 11008, 4096, 16, n=8, requests=11),
        case("bwd_ragged_321", "bwd", 321, 4096, 4096, 64, n=4, requests=9),
        # its adapter gradients, and those of a small micro-batch of many short samples
        case("grad_train_4096", "grad", 4096, 11008, 4096, 16, n=8, requests=11),
        case("grad_short_515", "grad", 515, 4096, 4096, 32, n=16, requests=40),
        # one layer input kept over the forward pass: a small one, and that of a long batch at the down projection
        case("ckpt_small_int8", "ckpt", 77, 1, 4096, 0),
        case("ckpt_long_e4m3", "ckpt", 8192, 1, 11008, 0, fmt="e4m3"),
        # the adapter gradients of one linear from such an input
        case("cgrad_513_int8", "cgrad", 513, 4096, 4096, 16),
        case("cgrad_4096_e4m3", "cgrad", 4096, 4096, 11008, 64, fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "grad", "ckpt", "cgrad"])
    fmt = rng.choice(["int8", "e4m3"])
    K = 64 * _log(rng, 1, 172)
    if op == "ckpt":
        return {"op": op, "M": _log(rng, 1, 8192), "N": 1, "K": K, "r": 0, "n": 1, "requests": 1, "fmt": fmt}
    # the forward takes any N; the gradients' rows are whole 16-byte pieces
    N = _log(rng, 40, 11008) if op == "fwd" else 8 * _log(rng, 5, 1376)
    M = _log(rng, 1 if op == "fwd" else 16, 4096)
    M = max(1, min(M, 4096 * 4096 * 11008 // (N * K)))
    r = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
    if op == "cgrad":
        return {"op": op, "M": M, "N": N, "K": K, "r": r, "n": 1, "requests": 1, "fmt": fmt}
    n = _log(rng, 1, 32)
    return {"op": op, "M": M, "N": N, "K": K, "r": r, "n": n, "requests": min(M, _log(rng, 1, 64)), "fmt": "int8"}


def work(case):
    op, M, N, K, r = (case[k] for k in ("op", "M", "N", "K", "r"))
    kept = M * K * (1 + 2 / BLOCK)                     # one byte a value and a bf16 a block
    if op == "ckpt":
        return {"bytes": 2 * M * K * 2 + 2 * kept, "flops": 0}
    if op == "cgrad":
        return {"bytes": kept + 2 * M * N + r * (K + N) * (2 + 4), "flops": 4 * M * r * (K + N)}
    used = len({q % case["n"] for q in range(case["requests"]) if q % 8 != 7})
    if op == "grad":
        return {"bytes": 2 * M * (K + N) + 4 * M + used * r * (K + N) * 2 + case["n"] * r * (K + N) * 4,
                "flops": 4 * M * r * (K + N)}
    weight = N * K * (0.5 + 1 / BLOCK + 4 / (BLOCK * GROUP))
    return {"bytes": weight + 2 * M * (K + N) + 4 * M + used * r * (K + N) * 2,
            "flops": 2 * M * N * K + 2 * M * r * (K + N)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, M, N, K, r, n = (case[k] for k in ("op", "M", "N", "K", "r", "n"))
    bf = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(bf)

    state = {"op": op, "M": M, "N": N, "K": K, "r": r, "n": n, "fmt": case["fmt"]}
    if op != "bwd":
        # layer inputs: unit normal with a few channels an order of magnitude larger
        gain = torch.ones(K, device=dev)
        gain[torch.randint(0, K, (max(1, K // 256),), generator=g, device=dev)] = 12.0
        x = (torch.randn(M, K, generator=g, device=dev) * gain).to(bf)
        if op == "cgrad":
            state["codes"], state["absmax"] = _keep(x, case["fmt"])
        else:
            state["x"] = x
    if op == "ckpt":
        return state
    if op != "fwd":
        state["dy"] = normal(M, N, std=1e-2)
    state["A"] = normal(n, r, K, std=K ** -0.5)
    state["B"] = normal(n, N, r, std=0.02)
    if op == "cgrad":
        state["alpha"] = 2.0 * r
        return state
    # alpha / r of each adapter
    state["scale"] = torch.rand(n, generator=g, device=dev) * 1.5 + 0.5
    # the batch: requests one after another, of uneven length; every eighth uses the base alone
    req = case["requests"]
    if req == M:
        lengths = torch.ones(M, dtype=torch.int64, device=dev)
    else:
        cuts = torch.sort(torch.randint(0, M + 1, (req - 1,), generator=g, device=dev)).values
        edge = torch.tensor([0], device=dev), cuts, torch.tensor([M], device=dev)
        lengths = torch.diff(torch.cat(edge))
    order = torch.randperm(n, generator=g, device=dev)
    q = torch.arange(req, device=dev)
    ids = torch.where(q % 8 == 7, -1, order[q % n])
    state["index"] = torch.repeat_interleave(ids, lengths, output_size=M).to(torch.int32)
    if op != "grad":
        # a stored weight of N(0, 0.02): the codes of such a weight are equally frequent
        nb = N * K // BLOCK
        ng = (nb + GROUP - 1) // GROUP
        state["packed"] = torch.randint(0, 256, (N * K // 2,), generator=g, device=dev, dtype=torch.uint8)
        state["qscale"] = torch.randint(70, 128, (nb,), generator=g, device=dev, dtype=torch.int8)
        state["step"] = (torch.rand(ng, generator=g, device=dev) * 0.2 + 0.9) * (0.07 / 127)
    return state


# --------------------------------------------------------------------------
# plain forms (32 bits)
# --------------------------------------------------------------------------
def _levels():
    # quantiles of N(0, 1) at (i + 1/2) / 16, divided by the largest; lower half mirrored
    p = (torch.arange(8, 16, dtype=torch.float64) + 0.5) / 16
    z = torch.special.ndtri(p)
    z = (z / z[-1]).float()
    return torch.cat([-z.flip(0), z])


def _weight(st):
    """W' [N, K] as 32-bit values of its bf16 entries."""
    p = st["packed"]
    L = _levels().to(p.device)
    codes = torch.stack([p & 15, p >> 4], dim=1).to(torch.int32)
    q = st["qscale"].float()
    d = st["step"].repeat_interleave(GROUP)[: q.numel()]
    w = L[codes].view(-1, BLOCK) * (q * d)[:, None]
    return w.to(torch.bfloat16).float().view(st["N"], st["K"])


def _top(fmt):
    return 127.0 if fmt == "int8" else 448.0


def _keep(x, fmt):
    """The 8-bit form of x: codes (int8 numbers or e4m3 bits) and the blocks' bf16 absmax."""
    v = x.float().view(-1, BLOCK)
    top = v.abs().amax(1, keepdim=True)
    f = torch.where(top > 0, v * _top(fmt) / top, 0.0)
    codes = f.round().to(torch.int8) if fmt == "int8" else f.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(x.shape), top.to(torch.bfloat16).view(-1)


def _kept(codes, absmax, fmt):
    """The bf16 values that a kept activation stands for."""
    v = codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    s = (absmax.double() / _top(fmt)).float()          # the correctly rounded quotient
    return (v.view(-1, BLOCK) * s[:, None]).to(torch.bfloat16).view(codes.shape)


def _spread(part, st):
    """part [M, n, r], kept where the row uses the adapter, times the adapter's scale: [M, n r]."""
    uses = st["index"].long()[:, None] == torch.arange(st["n"], device=part.device)
    return torch.where(uses[:, :, None], part * st["scale"][None, :, None], 0.0).view(part.shape[0], -1)


def _plain(st):
    op, M, N, K, r, n = (st[k] for k in ("op", "M", "N", "K", "r", "n"))
    if op == "ckpt":
        codes, absmax = _keep(st["x"], st["fmt"])
        return {"restored": _kept(codes, absmax, st["fmt"]), "absmax": absmax}
    A, B = st["A"].float(), st["B"].float()
    if op == "cgrad":
        x, dy = _kept(st["codes"], st["absmax"], st["fmt"]).float(), st["dy"].float()
        s = st["alpha"] / r
        return {"dA": (s * (dy @ B[0])).t() @ x, "dB": dy.t() @ (s * (x @ A[0].t()))}
    flatA, flatB = A.view(n * r, K), B.permute(0, 2, 1).reshape(n * r, N)
    if op == "fwd":
        x = st["x"].float()
        t = _spread((x @ flatA.t()).view(M, n, r), st)
        return (x @ _weight(st).t() + t @ flatB).to(torch.bfloat16)
    dy = st["dy"].float()
    u = _spread((dy @ flatB.t()).view(M, n, r), st)
    if op == "bwd":
        return (dy @ _weight(st) + u @ flatA).to(torch.bfloat16)
    x = st["x"].float()
    t = _spread((x @ flatA.t()).view(M, n, r), st)
    return {"dA": (u.t() @ x).view(n, r, K), "dB": (dy.t() @ t).view(N, n, r).permute(1, 0, 2).contiguous()}


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _handles(st):
    """What a program keeps for a layer: the stored weight, the pool of adapters, a workspace."""
    from qlora_dequant_gemm_amd import ops

    if "ws" not in st:
        st["ops"], st["ws"] = ops, ops.Workspace("cuda")
        if "packed" in st:
            st["qw"] = ops.NF4Weight(st["packed"], st["qscale"], st["step"], (st["N"], st["K"]))
        if "scale" in st:
            st["pool"] = ops.AdapterPool(st["A"], st["B"], st["scale"])
        if "codes" in st:
            st["kept"] = ops.Act8(st["codes"], st["absmax"], st["fmt"])
    return st["ops"]


def _own(st):
    ops = _handles(st)
    op = st["op"]
    if op == "ckpt":
        kept = ops.act8_pack(st["x"], st["fmt"])
        return {"restored": ops.act8_unpack(kept), "absmax": kept.absmax}
    if op == "cgrad":
        dA, dB = ops.lora_grad(st["kept"], st["dy"], st["A"][0], st["B"][0], st["alpha"], ws=st["ws"])
        return {"dA": dA, "dB": dB}
    if op == "fwd":
        return ops.lora_fwd_multi(st["x"], st["qw"], st["pool"], st["index"], ws=st["ws"])
    if op == "bwd":
        return ops.bwd_dx_multi(st["dy"], st["qw"], st["pool"], st["index"], ws=st["ws"])
    dA, dB = ops.lora_grad_multi(st["x"], st["dy"], st["pool"], st["index"], ws=st["ws"])
    return {"dA": dA, "dB": dB}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _round_e4m3(v):
    """Nearest e4m3 value of each |v| <= 448 (ties to even): steps of 2^(e-3), at least 2^-9."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step) * step


def _exact_kept(x, fmt):
    b = x.double().reshape(-1, 64)
    top = b.abs().max(dim=1).values
    live = top > 0
    v = b * _top(fmt) / torch.where(live, top, 1.0)[:, None]  # the product is exact
    v = torch.round(v) if fmt == "int8" else _round_e4m3(v)
    s = (top / _top(fmt)).float().double()             # the scale is a 32-bit number by definition
    return torch.where(live[:, None], v * s[:, None], 0.0).float().to(torch.bfloat16).reshape(x.shape), top


def _exact_weight(st):
    codes = torch.empty(st["N"] * st["K"], dtype=torch.long, device=st["packed"].device)
    codes[0::2], codes[1::2] = (st["packed"] % 16).long(), (st["packed"] // 16).long()
    block = torch.arange(codes.numel(), device=codes.device) // 64
    s = st["qscale"].double()[block] * st["step"].double()[block // 256]
    w = _levels().to(codes.device).double()[codes] * s.float().double()
    return w.float().to(torch.bfloat16).double().reshape(st["N"], st["K"])


def exact(case, seed):
    st = prepare(case, seed)
    op, n, r = st["op"], st["n"], st["r"]
    if op == "ckpt":
        restored, top = _exact_kept(st["x"], st["fmt"])
        return {"restored": restored.double(), "absmax": top}
    A, B = st["A"].double(), st["B"].double()
    if op == "cgrad":
        if st["fmt"] == "int8":
            v = st["codes"].double()
        else:
            bits = st["codes"].long()
            e, m = (bits >> 3) & 15, (bits & 7).double()
            v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
            v = torch.where(bits > 127, -v, v)
        s = (st["absmax"].double() / _top(st["fmt"])).float().double()
        x = (v.reshape(-1, 64) * s[:, None]).float().to(torch.bfloat16).double().reshape(st["M"], st["K"])
        groups = [(0, slice(None), st["alpha"] / r)]
    else:
        x = st["x"].double() if "x" in st else None
        groups = [(a, torch.nonzero(st["index"] == a)[:, 0], st["scale"][a].double()) for a in range(n)]
    dy = st["dy"].double() if "dy" in st else None
    if op == "fwd":
        y = x @ _exact_weight(st).t()
        for a, rows, s in groups:
            y[rows] += s * ((x[rows] @ A[a].t()) @ B[a].t())
        return y
    if op == "bwd":
        dx = dy @ _exact_weight(st)
        for a, rows, s in groups:
            dx[rows] += s * ((dy[rows] @ B[a]) @ A[a])
        return dx
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a, rows, s in groups:
        dA[a] = s * ((dy[rows] @ B[a]).t() @ x[rows])
        dB[a] = s * (dy[rows].t() @ (x[rows] @ A[a].t()))
    return {"dA": dA[0], "dB": dB[0]} if op == "cgrad" else {"dA": dA, "dB": dB}
