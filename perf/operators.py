"""The training operators around the routed experts, as measured cases.

Three operators, each forwards and backwards where it has both:
  sort / unsort    tokens moved to expert-sorted rows and back, weights applied, with both gradients
  checkpoint       the combine that leaves an 8-bit checkpoint of the expert outputs, and its backward from it
  router           the gradient through gates, sigmoid, balance loss and the logits product

With ``own`` false, run() computes them with elementary torch operations in
32 bits; with ``own`` true it makes the calls of this repository's package.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one decoded token goes to its eight experts: latency alone
        dict(name="sort_one_token", op="sort", dir="fwd", T=1, K=8, E=256, d=7168, type="bf16", drop=0.0, pad=0),
        # gradient of the sorted tokens of a prefill-sized training batch
        dict(name="sort_bwd_prefill", op="sort", dir="bwd", T=4096, K=8, E=256, d=7168, type="bf16", drop=0.0, pad=0),
        # a padded batch of odd width in half precision, rows of a wider buffer, pairs dropped
        dict(name="unsort_odd_padded", op="unsort", dir="fwd", T=1021, K=6, E=40, d=1111, type="fp16", drop=0.15, pad=9),
        # a small fine-tuning batch in 32 bits: gradients of rows and weights
        dict(name="unsort_bwd_small", op="unsort", dir="bwd", T=256, K=8, E=256, d=7168, type="fp32", drop=0.0, pad=0),
        # the largest batch of the layer's shapes: gradients of rows and weights
        dict(name="unsort_bwd_large", op="unsort", dir="bwd", T=16384, K=6, E=384, d=7168, type="bf16", drop=0.0, pad=0),
        # combine and checkpoint of a small batch
        dict(name="checkpoint_small", op="checkpoint", dir="fwd", T=256, K=8, E=256, d=7168, pow2=False, drop=0.0),
        # combine and checkpoint of a prefill-sized training batch
        dict(name="checkpoint_prefill", op="checkpoint", dir="fwd", T=4096, K=8, E=256, d=7168, pow2=False, drop=0.0),
        # its backward: FP8 gradient rows and the gates' gradient
        dict(name="checkpoint_bwd_prefill", op="checkpoint", dir="bwd", T=4096, K=8, E=256, d=7168, pow2=False, drop=0.0),
        # an odd batch with dropped pairs and power-of-two scales
        dict(name="checkpoint_bwd_odd", op="checkpoint", dir="bwd", T=333, K=6, E=40, d=1152, pow2=True, drop=0.1),
        # a small fine-tuning batch without the balance loss
        dict(name="router_small", op="router", dir="bwd", T=200, K=8, E=256, d=7168, n_seq=0),
        # prefill-sized training batch, four sequences with the balance loss
        dict(name="router_prefill", op="router", dir="bwd", T=4096, K=8, E=256, d=7168, n_seq=4),
        # the largest batch and expert count of the layer's shapes
        dict(name="router_large", op="router", dir="bwd", T=16384, K=6, E=384, d=7168, n_seq=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "sort", "unsort", "unsort", "checkpoint", "checkpoint", "router", "router"])
    K = rng.choice([1, 2, 4, 6, 8])
    if op in ("sort", "unsort"):
        d = rng.choice([_log(rng, 64, 7168), 8 * _log(rng, 8, 896), 7168])
        T = min(_log(rng, 1, 16384), 16384 * 6 * 7168 // (2 * K * d))
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, K=K, E=rng.choice([16, 40, 64, 256, 384]), d=d,
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), drop=rng.choice([0.0, 0.0, 0.1, 0.5]),
                    pad=rng.choice([0, 0, 8, 5]))
    if op == "checkpoint":
        d = 128 * _log(rng, 1, 56)
        T = _log(rng, 1, 4096)
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, K=K, E=rng.choice([16, 40, 64, 256, 384]), d=d,
                    pow2=rng.choice([False, True]), drop=rng.choice([0.0, 0.0, 0.2]))
    n_seq = rng.choice([0, 1, 3, 8])
    T = _log(rng, 8, 16384)
    if n_seq:
        T = max(1, T // (8 * n_seq)) * 8 * n_seq
    return dict(op=op, dir="bwd", T=T, K=K, E=16 * rng.choice([1, 3, 4, 5, 8, 16, 24]), d=128 * _log(rng, 1, 56), n_seq=n_seq)


# ------------------------------------------------------------------ inputs --
def _rows(gen, n, d, std, type_="fp32", pad=0):
    """N(0, std^2) rows with a few outlying values, as a view of rows of d + pad elements."""
    x = torch.randn(n, d + pad, generator=gen, device=DEV) * std
    x[:, ::61] *= 1.0 + 8.0 * (torch.rand(n, 1, generator=gen, device=DEV) < 0.05)
    return x.to(TYPES[type_])[:, :d]


def _kept(case):
    """Pairs that are not dropped."""
    P = case["T"] * case["K"]
    return P - int(P * case.get("drop", 0.0))


def _routing(gen, case):
    """Top-K of a skewed router: (idx, gate, dst_of, kept pairs); dropped pairs have dst_of -1."""
    T, K, E = case["T"], case["K"], case["E"]
    z = torch.randn(T, E, generator=gen, device=DEV) + 0.7 * torch.randn(E, generator=gen, device=DEV)
    s = torch.sigmoid(z)
    top, idx = s.topk(K, dim=1)
    gate = top / top.sum(1, keepdim=True)
    n = _kept(case)
    keep = (torch.rand(T * K, generator=gen, device=DEV).argsort() < n).view(T, K)
    key = torch.where(keep, idx, E).reshape(-1)
    order = torch.argsort(key, stable=True)
    dst = torch.empty(T * K, dtype=torch.int64, device=DEV)
    dst[order] = torch.arange(T * K, device=DEV)
    dst = torch.where(keep, dst.view(T, K), -1).to(torch.int32)
    return idx.to(torch.int32), gate, dst, n


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7919 * seed + 13)
    op, T, K, d = case["op"], case["T"], case["K"], case["d"]
    s = dict(case=case)
    if op in ("sort", "unsort"):
        _, s["gate"], s["dst"], n = _routing(gen, case)
        tok, srt = _rows(gen, T, d, 1.0, case["type"], case["pad"]), None
        if (op, case["dir"]) != ("sort", "fwd"):
            srt = _rows(gen, n, d, 1.0, case["type"], case["pad"])
        s.update(tok=tok, srt=srt, n=n)
    elif op == "checkpoint":
        _, s["gate"], s["dst"], n = _routing(gen, case)
        s["n"] = n
        y = _rows(gen, n, d, 0.5)
        if case["dir"] == "fwd":
            s.update(y=y, y_shared=_rows(gen, T, d, 0.5), u=_rows(gen, T, d, 1.0, "bf16"))
        else:
            q, sc = _quant(y, case["pow2"])
            s.update(dout=_rows(gen, T, d, 0.01), yq=q.view(torch.uint8), ys=sc)
            # the program's own gradient buffers: a row that no pair points at keeps what it held
            s["dyq"] = torch.zeros(T * K + T, d, dtype=torch.uint8, device=DEV)
            s["dys"] = torch.zeros(T * K + T, d // 128, device=DEV)
    else:
        E = case["E"]
        u = torch.randn(T, d, generator=gen, device=DEV).to(torch.bfloat16)
        cent = (torch.randn(E, d, generator=gen, device=DEV) / math.sqrt(d)).to(torch.bfloat16)
        bias = 0.1 * torch.rand(E, generator=gen, device=DEV)
        z = u.float() @ cent.float().T
        a = torch.sigmoid(z)
        idx = (a + bias).topk(K, dim=1).indices
        top = a.gather(1, idx)
        s.update(u=u, cent=cent, z=z, idx=idx.to(torch.int32), gate=top / top.sum(1, keepdim=True),
                 dgate=0.1 * torch.randn(T, K, generator=gen, device=DEV),
                 base=1e-3 * torch.randn(T, d, generator=gen, device=DEV), f=None, dloss=None, alpha=1e-4)
        if case["n_seq"]:
            S = T // case["n_seq"]
            member = torch.zeros(T, E, device=DEV).scatter_(1, a.topk(K, dim=1).indices, 1.0)
            s["f"] = member.view(-1, S, E).sum(1) * (E / (K * S))
            s["dloss"] = 0.5 + torch.rand(case["n_seq"], generator=gen, device=DEV)
    return s


# -------------------------------------------------------------- plain forms --
def _quant(x, pow2):
    """1x128 E4M3 quantisation of fp32 rows: (codes as float8 values, scales)."""
    n, d = x.shape
    t = x.view(n, d // 128, 128)
    top = t.abs().amax(2).clamp_min(1e-4)
    sc = top / torch.full_like(top, 448.0)          # by a tensor: a division, not a product with 1/448
    if pow2:
        b = sc.view(torch.int32)
        sc = torch.where((b & 0x7FFFFF) != 0, (b & 0x7F800000) + 0x800000, b).view(torch.float32)
    q = (t / sc[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(n, d), sc


def _pairs(dst):
    """(token, slot, row) of the kept pairs."""
    t, k = torch.nonzero(dst >= 0, as_tuple=True)
    return t, k, dst[t, k].long()


def _plain_sort(s):
    c, dst = s["case"], s["dst"]
    if c["dir"] == "fwd":
        t, _, r = _pairs(dst)
        out = torch.empty(s["n"], c["d"], dtype=s["tok"].dtype, device=DEV)
        out[r] = s["tok"][t]
        return out
    rows = s["srt"].float()[dst.clamp_min(0).long()] * (dst >= 0)[:, :, None]
    return rows.sum(1).to(s["srt"].dtype)


def _plain_unsort(s):
    c, dst, gate, y = s["case"], s["dst"], s["gate"], s["srt"]
    w = torch.where(dst >= 0, gate, 0.0)
    safe = dst.clamp_min(0).long()
    if c["dir"] == "fwd":
        return (y.float()[safe] * w[:, :, None]).sum(1).to(y.dtype)
    t, k, r = _pairs(dst)
    dout = s["tok"].float()
    dy = torch.zeros(s["n"], c["d"], dtype=y.dtype, device=DEV)
    dy[r] = (gate[t, k][:, None] * dout[t]).to(y.dtype)
    dw = torch.zeros_like(gate)
    dw[t, k] = (dout[t] * y.float()[r]).sum(1)
    return dy, dw


def _plain_checkpoint(s):
    c, dst, gate = s["case"], s["dst"], s["gate"]
    safe, keep = dst.clamp_min(0).long(), dst >= 0
    if c["dir"] == "fwd":
        w = torch.where(keep, gate, 0.0)
        out = s["u"].float() + s["y_shared"] + (s["y"][safe] * w[:, :, None]).sum(1)
        q, sc = _quant(s["y"], c["pow2"])
        return out, q, sc
    t, k, r = _pairs(dst)
    T, P = c["T"], c["T"] * c["K"]
    dout = s["dout"]
    q, sc = torch.zeros_like(s["dyq"]).view(torch.float8_e4m3fn), torch.zeros_like(s["dys"])
    routed, routed_scale = _quant(gate[t, k][:, None] * dout[t], True)
    q.view(torch.uint8)[r], sc[r] = routed.view(torch.uint8), routed_scale
    q[P:], sc[P:] = _quant(dout, True)
    y = (s["yq"].view(torch.float8_e4m3fn).float().view(s["n"], -1, 128) * s["ys"][:, :, None]).view(s["n"], -1)
    dgate = torch.zeros_like(gate)
    dgate[t, k] = (dout[t] * y[r]).sum(1)
    return q, sc, dgate


def _plain_router(s):
    c, z, g = s["case"], s["z"], s["gate"]
    a, rest = torch.sigmoid(z), torch.sigmoid(-z)
    idx = s["idx"].long()
    dz = torch.zeros_like(z)
    dz.scatter_add_(1, idx, g * rest.gather(1, idx) * (s["dgate"] - (g * s["dgate"]).sum(1, keepdim=True)))
    if s["f"] is not None:
        S = c["T"] // c["n_seq"]
        cost = (s["f"] * (s["alpha"] * s["dloss"] / S)[:, None]).repeat_interleave(S, 0)
        norm = a / a.sum(1, keepdim=True)
        dz += norm * rest * (cost - (norm * cost).sum(1, keepdim=True))
    return dz, s["base"] + dz @ s["cent"].float(), dz.T @ s["u"].float()


# ---------------------------------------------------------- the own kernels --
def _own(s):
    import fp8_block_scaled_sigmoid_b200 as moe
    c = s["case"]
    op, fwd = c["op"], c["dir"] == "fwd"
    if op == "sort":
        if fwd:
            return moe.moe_sort_rows(s["tok"], s["dst"], s["n"])
        return moe.moe_sort_rows_backward(s["srt"], s["dst"])
    if op == "unsort":
        if fwd:
            return moe.moe_unsort_rows(s["srt"], s["dst"], s["gate"])
        return moe.moe_unsort_rows_backward(s["tok"], s["srt"], s["dst"], s["gate"])
    f8 = torch.float8_e4m3fn
    if op == "checkpoint":
        if fwd:
            out, q, sc = moe.moe_combine_checkpoint(s["y"], s["dst"], s["gate"], s["y_shared"], s["u"], pow2=c["pow2"])
            return out, q.view(f8), sc
        q, sc, _, dgate = moe.moe_combine_checkpoint_backward(s["dout"], s["dst"], s["gate"], s["yq"], s["ys"],
                                                              dyq=s["dyq"], dys=s["dys"])
        return q.view(f8), sc, dgate
    return moe.moe_route_backward(s["dgate"], s["z"], s["idx"], s["gate"], s["u"], s["cent"], du_base=s["base"],
                                  f=s["f"], dloss=s["dloss"], alpha=s["alpha"],
                                  seq_len=c["T"] // c["n_seq"] if c["n_seq"] else 0)


def run(state):
    if own:
        return _own(state)
    return {"sort": _plain_sort, "unsort": _plain_unsort, "checkpoint": _plain_checkpoint,
            "router": _plain_router}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work --
def work(case):
    op, T, K, d = case["op"], case["T"], case["K"], case["d"]
    fwd = case["dir"] == "fwd"
    P = _kept(case)
    if op in ("sort", "unsort"):
        e = SIZE[case["type"]]
        rows = T + P if op == "sort" or fwd else T + 2 * P
        table = T * K * 4 * (1 if op == "sort" else (2 if fwd else 3))
        flops = 0 if (op, fwd) == ("sort", True) else P * d * (1 if op == "sort" else (2 if fwd else 3))
        return {"bytes": rows * d * e + table, "flops": flops}
    q = 1.0 + 4.0 / 128.0
    if op == "checkpoint":
        if fwd:
            return {"bytes": P * d * 4 + T * d * 10 + P * d * q + T * K * 8, "flops": P * d * 4}
        return {"bytes": T * d * 4 + P * d * q + (P + T) * d * q + T * K * 12, "flops": P * d * 5}
    E = case["E"]
    return {"bytes": T * E * 8 + T * d * 10 + E * d * 6 + T * K * 12, "flops": 4.0 * T * E * d}


# ------------------------------------------------------------------- exact --
def _e4m3(v):
    """Nearest E4M3 value (ties to even, saturating at 448) of 64-bit numbers."""
    a = v.abs().clamp_max(448.0)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    e = torch.where(a < torch.exp2(e), e - 1, e)          # log2 rounded up over a power of two
    e = torch.where(a >= torch.exp2(e + 1), e + 1, e).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.copysign(torch.round(a / step) * step, v)


def _exact_quant(v, pow2):
    """Codes' values and scales of 64-bit rows that hold 32-bit numbers: the scale and the quotient each rounded once to 32 bits."""
    n, d = v.shape
    t = v.view(n, d // 128, 128)
    floor = torch.tensor(1e-4, dtype=torch.float32, device=v.device).double()
    sc = (torch.maximum(t.abs().amax(2), floor) / 448.0).float().double()
    if pow2:
        m, e = torch.frexp(sc)
        sc = torch.ldexp(torch.ones_like(sc), torch.where(m == 0.5, e - 1, e))
    return _e4m3((t / sc[:, :, None]).float().double()).view(n, d), sc


def _exact_tokens(s, lo, hi):
    """The outputs of tokens lo..hi by the definition, in 64 bits."""
    c = s["case"]
    dst = s["dst"][lo:hi].long()
    keep, safe = dst >= 0, dst.clamp_min(0)
    gate = s["gate"][lo:hi].double() * keep
    if c["op"] == "checkpoint":
        return s["u"][lo:hi].double() + s["y_shared"][lo:hi].double() + torch.einsum("tk,tkd->td", gate, s["y"][safe].double())
    weight = gate if c["op"] == "unsort" else keep.double()
    return torch.einsum("tk,tkd->td", weight, s["srt"][safe].double())


def _source(dst, n):
    """For each sorted row its token and slot."""
    T, K = dst.shape
    flat = torch.empty(n, dtype=torch.int64, device=dst.device)
    where = torch.nonzero(dst.reshape(-1) >= 0).reshape(-1)
    flat[dst.reshape(-1)[where].long()] = where
    return flat // K, flat % K


def exact(case, seed):
    s = prepare(case, seed)
    op, T, K, d = case["op"], case["T"], case["K"], case["d"]
    step = max(1, (1 << 26) // (K * d))
    chunks = [(i, min(T, i + step)) for i in range(0, T, step)]
    rows = [(i, min(s["n"], i + step * K)) for i in range(0, s["n"], step * K)] if "n" in s else []
    if op == "router":
        z, g, dg = s["z"].double(), s["gate"].double(), s["dgate"].double()
        inv = 1.0 / (1.0 + torch.exp(z))                   # 1 - sigmoid(z)
        a = 1.0 / (1.0 + torch.exp(-z))
        ds = dg - torch.einsum("tk,tk->t", g, dg)[:, None]
        onehot = torch.zeros(T, case["E"], dtype=torch.float64, device=DEV)
        onehot.scatter_add_(1, s["idx"].long(), g * ds)
        dz = onehot * inv
        if s["f"] is not None:
            S = T // case["n_seq"]
            p = a / a.sum(1, keepdim=True)
            cost = s["alpha"] / S * s["dloss"].double()[:, None] * s["f"].double()
            cost = cost[torch.arange(T, device=DEV) // S]
            dz = dz + p * inv * (cost - torch.einsum("te,te->t", p, cost)[:, None])
        return dz, s["base"].double() + dz @ s["cent"].double(), dz.T @ s["u"].double()
    if op in ("sort", "unsort"):
        if case["dir"] == "fwd" and op == "sort":
            t, _ = _source(s["dst"], s["n"])
            return s["tok"][t].double()
        if case["dir"] == "bwd" and op == "unsort":
            t, k = _source(s["dst"], s["n"])
            dy = torch.empty(s["n"], d, dtype=torch.float64, device=DEV)
            dw = torch.zeros(T, K, dtype=torch.float64, device=DEV)
            for i, j in rows:
                dout = s["tok"][t[i:j]].double()
                dy[i:j] = s["gate"][t[i:j], k[i:j]].double()[:, None] * dout
                dw[t[i:j], k[i:j]] = torch.einsum("rd,rd->r", dout, s["srt"][i:j].double())
            return dy, dw
        return torch.cat([_exact_tokens(s, a, b) for a, b in chunks])
    if case["dir"] == "fwd":
        q, sc = _exact_quant(s["y"].double(), case["pow2"])
        return torch.cat([_exact_tokens(s, a, b) for a, b in chunks]), q, sc
    q = torch.zeros(T * K + T, d, dtype=torch.float32, device=DEV)
    sc = torch.zeros(T * K + T, d // 128, dtype=torch.float64, device=DEV)
    t, k = _source(s["dst"], s["n"])
    dgate = torch.zeros(T, K, dtype=torch.float64, device=DEV)
    for i, j in rows:
        dout = s["dout"][t[i:j]].double()
        q[i:j], sc[i:j] = _exact_quant((s["gate"][t[i:j], k[i:j]].double()[:, None] * dout).float().double(), True)
        y = s["yq"][i:j].view(torch.float8_e4m3fn).double().view(j - i, -1, 128) * s["ys"][i:j].double()[:, :, None]
        dgate[t[i:j], k[i:j]] = torch.einsum("rd,rd->r", dout, y.view(j - i, d))
    q[T * K:], sc[T * K:] = _exact_quant(s["dout"].double(), True)
    return q, sc, dgate
