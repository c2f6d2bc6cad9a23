"""Cases that measure the mixture-of-experts operators of the package.

A mixture-of-experts layer with INT4 weights routes each token to a few
experts.  Its operators, and the gradients that a training step takes through
them while the packed weights stay frozen:

  sort              tokens gathered into the order of their experts
  combine           the experts' rows back to their tokens, weighted and summed
                    (without weights it is the gradient of sort)
  combine_backward  its gradients: of the experts' rows and of the weights
  gemm              each expert's rows times that expert's INT4 weights
  gemm_dx           the gradient of that product with respect to its rows

`own` selects between the plain form (elementary torch operations in 32 bits)
and the package's operators; `exact` computes the definition in 64 bits.
"""
import torch

own = False

GROUPS = (-1, 32, 64, 128)


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one token of a chat: launch latency
        {"name": "sort 1 token", "op": "sort", "tokens": 1, "topk": 8, "experts": 64,
         "hidden": 2048, "drop": 0.0},
        # a long prompt on one rank of an expert-parallel pair: half of the
        # chosen experts live on the other rank
        {"name": "sort 8192 tokens", "op": "sort", "tokens": 8192, "topk": 2, "experts": 8,
         "hidden": 5120, "drop": 0.5},
        # a small batch being decoded
        {"name": "combine 8 tokens", "op": "combine", "tokens": 8, "topk": 8, "experts": 64,
         "hidden": 2048, "weighted": True, "drop": 0.0},
        # a prompt through many small experts
        {"name": "combine 4096 tokens", "op": "combine", "tokens": 4096, "topk": 8,
         "experts": 64, "hidden": 2048, "weighted": True, "drop": 0.0},
        # a short, odd fine-tuning batch
        {"name": "combine_backward 37 tokens", "op": "combine_backward", "tokens": 37, "topk": 3,
         "experts": 12, "hidden": 1048, "weighted": True, "drop": 0.1},
        # a full fine-tuning batch
        {"name": "combine_backward 8192 tokens", "op": "combine_backward", "tokens": 8192,
         "topk": 2, "experts": 8, "hidden": 5120, "weighted": True, "drop": 0.0},
        # one token through its eight experts' up-projections
        {"name": "gemm 1 token", "op": "gemm", "tokens": 1, "topk": 8, "experts": 64, "K": 2048,
         "N": 2048, "group": 128, "drop": 0.0},
        # a serving batch: a few rows for every expert
        {"name": "gemm 64 tokens", "op": "gemm", "tokens": 64, "topk": 8, "experts": 64,
         "K": 2048, "N": 2048, "group": 32, "drop": 0.0},
        # a prompt with ragged row counts and odd sizes
        {"name": "gemm 1001 tokens", "op": "gemm", "tokens": 1001, "topk": 6, "experts": 48,
         "K": 1424, "N": 2056, "group": 64, "drop": 0.05},
        # a long prompt through a few large experts
        {"name": "gemm 4096 tokens", "op": "gemm", "tokens": 4096, "topk": 2, "experts": 8,
         "K": 5120, "N": 17408, "group": 128, "drop": 0.0},
        # a fine-tuning step over many small experts
        {"name": "gemm_dx 1024 tokens", "op": "gemm_dx", "tokens": 1024, "topk": 8,
         "experts": 64, "K": 2048, "N": 2048, "group": 128, "drop": 0.0},
        # a fine-tuning step over a few large experts' down-projections
        {"name": "gemm_dx 2048 tokens", "op": "gemm_dx", "tokens": 2048, "topk": 2,
         "experts": 8, "K": 17408, "N": 5120, "group": 32, "drop": 0.0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("sort", "combine", "combine_backward", "gemm", "gemm", "gemm_dx"))
    while True:
        case = {"op": op, "tokens": _log_uniform(rng, 1, 8192)}
        case["experts"] = _log_uniform(rng, 2, 128)
        case["topk"] = min(rng.choice((1, 2, 3, 4, 6, 8)), case["experts"])
        case["drop"] = rng.choice((0.0, 0.0, 0.1, 0.5))
        if op in ("gemm", "gemm_dx"):
            case["K"] = 16 * _log_uniform(rng, 8, 1088)
            case["N"] = 8 * _log_uniform(rng, 16, 2176)
            case["group"] = rng.choice(GROUPS)
            rows = case["tokens"] * case["topk"]
            if (case["experts"] * case["K"] * case["N"] <= 8 * 5120 * 17408
                    and rows * case["K"] * case["N"] <= 8192 * 5120 * 17408 // 2
                    and rows * (case["K"] + case["N"]) <= 8192 * (5120 + 17408)):
                return case
        else:
            case["hidden"] = 8 * _log_uniform(rng, 8, 1024)
            if op != "sort":
                case["weighted"] = op == "combine_backward" or rng.random() < 0.7
            if case["tokens"] * case["topk"] * case["hidden"] <= 8192 * 2 * 5120:
                return case


def _rows(case):
    return case["tokens"] * case["topk"]


def _scale_rows(K, group):
    return 1 if group == -1 or group >= K else -(-K // group)


def _live_rows(case):
    """Expected rows after dropping."""
    return max(1.0, _rows(case) * (1.0 - case["drop"]))


def work(case):
    m, topk, op = case["tokens"], case["topk"], case["op"]
    live = _live_rows(case)
    if op in ("gemm", "gemm_dx"):
        K, N, E = case["K"], case["N"], case["experts"]
        used = E * (1.0 - (1.0 - 1.0 / E) ** live) if m > 1 else min(E, live)
        weights = used * (K * N / 2 + _scale_rows(K, case["group"]) * N * 2)
        return {"bytes": weights + live * (K + N) * 2, "flops": 2.0 * live * K * N}
    h = case["hidden"]
    if op == "sort":
        return {"bytes": 2 * h * (m + live) + 8 * _rows(case) + 4 * (case["experts"] + 1),
                "flops": 0}
    if op == "combine":
        return {"bytes": 2 * h * (m + live) + (8 if case["weighted"] else 4) * _rows(case),
                "flops": 2.0 * live * h}
    return {"bytes": 2 * h * (m + 2 * live) + 12 * _rows(case), "flops": 3.0 * live * h}


# ---- inputs ------------------------------------------------------------------

def _routing(case, gen):
    """Expert ids [tokens, topk] (int32, -1 where dropped) from router scores
    with a bias per expert, and the softmax weights of the chosen ones."""
    dev = "cuda"
    m, E, topk = case["tokens"], case["experts"], case["topk"]
    scores = torch.randn(m, E, generator=gen, device=dev)
    scores += 0.5 * torch.randn(E, generator=gen, device=dev)
    top, ids = scores.topk(topk, dim=1)
    dropped = torch.rand(m, topk, generator=gen, device=dev) < case["drop"]
    if m * topk > 0:
        dropped.view(-1)[0] = False
    ids = torch.where(dropped, torch.full_like(ids, -1), ids).to(torch.int32)
    return ids.contiguous(), torch.softmax(top, dim=1).contiguous()


def _placement(ids, E):
    """Row of each (token, choice) in expert order (int32, -1 where dropped),
    and the experts' first rows [E + 1]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    dest = torch.empty_like(order)
    dest[order] = torch.arange(order.numel(), device=ids.device)
    dest = torch.where(key < E, dest, torch.full_like(dest, -1))
    return order, offsets.to(torch.int32), dest.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f16 = dict(device="cuda", dtype=torch.float16)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.float16)

    st = {"case": dict(case)}
    ids, weights = _routing(case, gen)
    m, rows, E = case["tokens"], _rows(case), case["experts"]
    _, offsets, dest = _placement(ids, E)
    op = case["op"]
    if op in ("gemm", "gemm_dx"):
        K, N = case["K"], case["N"]
        words = torch.randint(-2 ** 31, 2 ** 31, (E, K // 8, N), generator=gen, device="cuda",
                              dtype=torch.int32)
        scales = torch.empty(E, _scale_rows(K, case["group"]), N, device="cuda")
        scales.uniform_(1e-3, 2e-2, generator=gen)
        st.update(offsets=offsets, qweight=words, scales=scales.to(torch.float16))
        # rows behind the last expert's keep what the output buffer holds
        if op == "gemm":
            st.update(x=normal(rows, K), out=torch.zeros(rows, N, **f16))
        else:
            st.update(x=normal(rows, N), out=torch.zeros(rows, K, **f16))
        return st
    h = case["hidden"]
    if op == "sort":
        st.update(x=normal(m, h), ids=ids, out=torch.zeros(rows, h, **f16))
        return st
    st.update(y=normal(rows, h), dest=dest, weights=weights if case["weighted"] else None)
    if op == "combine":
        st.update(out=torch.zeros(m, h, **f16))
    else:
        st.update(dout=normal(m, h), out=torch.zeros(rows, h, **f16))
    return st


# ---- one pass ------------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import int4_weight_only_gptq_b200 as pkg
    case = st["case"]
    op = case["op"]
    if op == "sort":
        return pkg.moe_sort(st["x"], st["ids"], case["experts"], out=st["out"])
    if op == "combine":
        return pkg.moe_combine(st["y"], st["dest"], st["weights"], out=st["out"])
    if op == "combine_backward":
        return pkg.moe_combine_backward(st["dout"], st["y"], st["dest"], st["weights"],
                                        out=st["out"])
    product = pkg.gemm_experts if op == "gemm" else pkg.gemm_experts_dx
    return product(st["x"], st["qweight"], st["scales"], st["offsets"], case["group"],
                   out=st["out"])


def _dequant(words, scales, K, group):
    """One expert's weights [K, N]: (q - 8) * scale rounded to FP16, in FP32."""
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    codes = (words[:, None, :] >> shifts[None, :, None]) & 15
    codes = (codes - 8).reshape(K, -1).float()
    if group == -1 or group >= K:
        return (codes * scales.float()).half().float()
    k_group = torch.arange(K, device=words.device) // group
    return (codes * scales.float()[k_group]).half().float()


def _run_plain(st):
    case = st["case"]
    op, E, topk = case["op"], case["experts"], case["topk"]
    out = st["out"]
    if op == "sort":
        order, offsets, dest = _placement(st["ids"], E)
        live = torch.arange(order.numel(), device=order.device) < offsets[E]
        out.copy_(torch.where(live[:, None], st["x"][order // topk], out))
        return out, offsets, dest
    if op == "combine":
        dest = st["dest"].long()
        sums = torch.zeros(out.shape, device=out.device)
        for j in range(topk):
            there = dest[:, j] >= 0
            rows = st["y"][dest[:, j].clamp(min=0)].float()
            if st["weights"] is not None:
                rows = rows * st["weights"][:, j, None]
            sums = sums + torch.where(there[:, None], rows, torch.zeros_like(rows))
        out.copy_(sums)
        return out
    if op == "combine_backward":
        dest, weights, dout = st["dest"].long(), st["weights"], st["dout"].float()
        dw = torch.zeros_like(weights)
        scratch = torch.cat([out, out[:1]])  # the last row takes what is dropped
        for j in range(topk):
            there = dest[:, j] >= 0
            rows = st["y"][dest[:, j].clamp(min=0)].float()
            dw[:, j] = torch.where(there, (rows * dout).sum(dim=1), 0.0)
            scratch[torch.where(there, dest[:, j], out.shape[0])] = (
                weights[:, j, None] * dout).half()
        out.copy_(scratch[:-1])
        return out, dw
    K, group = case["K"], case["group"]
    bounds = st["offsets"].tolist()
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            w = _dequant(st["qweight"][e], st["scales"][e], K, group)
            out[lo:hi] = st["x"][lo:hi].float() @ (w if op == "gemm" else w.T)
    return out


# ---- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op, E, topk = case["op"], case["experts"], case["topk"]
    if op == "sort":
        ids = st["ids"].reshape(-1).cpu().tolist()
        chosen = [[] for _ in range(E)]
        for pair, e in enumerate(ids):
            if 0 <= e < E:
                chosen[e].append(pair)
        out = st["out"].double()
        pairs = [p for lst in chosen for p in lst]
        if pairs:
            tokens = torch.tensor(pairs, device="cuda") // topk
            out[:len(pairs)] = st["x"].double()[tokens]
        offsets, dest = [0], [-1] * len(ids)
        for lst in chosen:
            offsets.append(offsets[-1] + len(lst))
        for row, p in enumerate(pairs):
            dest[p] = row
        return (out, torch.tensor(offsets, dtype=torch.int32),
                torch.tensor(dest, dtype=torch.int32).view(st["ids"].shape))
    if op in ("combine", "combine_backward"):
        # rows back to tokens as one indexed sum over the pairs that are kept
        flat = st["dest"].reshape(-1).long()
        pairs = torch.nonzero(flat >= 0).reshape(-1)
        tokens, rows = pairs // topk, flat[pairs]
        w = (torch.ones(flat.numel(), device="cuda", dtype=torch.float64)
             if st["weights"] is None else st["weights"].reshape(-1).double())
        y = st["y"].double()
        if op == "combine":
            out = torch.zeros(st["out"].shape, device="cuda", dtype=torch.float64)
            out.index_add_(0, tokens, y[rows] * w[pairs, None])
            return out
        dout = st["dout"].double()
        dy = st["out"].double()
        dy[rows] = dout[tokens] * w[pairs, None]
        dw = torch.zeros(flat.numel(), device="cuda", dtype=torch.float64)
        dw[pairs] = torch.einsum("ph,ph->p", dout[tokens], y[rows])
        return dy, dw.view(st["weights"].shape)
    K, N, group = case["K"], case["N"], case["group"]
    out = st["out"].double()
    bounds = st["offsets"].tolist()
    span = K if group == -1 else group
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        w = torch.empty(K, N, device="cuda", dtype=torch.float64)
        for j in range(8):
            w[j::8] = ((st["qweight"][e].long() >> (4 * j)) % 16 - 8).double()
        for g, k0 in enumerate(range(0, K, span)):
            w[k0:k0 + span] *= st["scales"][e, g].double()
        w = w.half().double()  # the definition rounds each weight to FP16
        rows = st["x"][lo:hi].double()
        out[lo:hi] = rows @ w if op == "gemm" else rows @ w.T
    return out
