"""Cases of the router, of the expert layer for few tokens, and of its weights in 4 bits: inputs, plain forms, the
library's calls.

Four operators:
  route    router scores to the chosen experts and their gates (forward), and the gates' gradient to the scores
  ffn      the whole gated expert layer for few tokens, weights in bfloat16, float32 or 4 bits
  project  one expert projection for few tokens: matrix-vector products, weights in bfloat16, float32 or 4 bits
  weights  an expert weight tensor into 4 bits and back

4-bit weights: every G input rows of a column share a bfloat16 scale, the value is code * scale with codes in [-8, 7].
The codes of input rows 8j .. 8j+7 of a column are one 32-bit word: row 8j+i as code + 8 at bit 4 * (i // 2) + 16 * (i % 2).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = torch.finfo(torch.float32).max


def listed():
    return [
        # decoding: one token of each of 8 ranks through the large layer's router, where the call's latency counts
        dict(name="route_decode", op="route", part="forward", R=8, S=1, E=256, K=8, score="sigmoid", renorm=True,
             bias=True, scale=2.5),
        # training: the large layer's router, sigmoid scores, the choice corrected by a bias per expert
        dict(name="route_large", op="route", part="forward", R=8, S=4096, E=256, K=8, score="sigmoid", renorm=True,
             bias=True, scale=2.5),
        # training: the mid layer's router, softmax over all experts, backward
        dict(name="route_back_mid", op="route", part="backward", R=8, S=4096, E=64, K=6, score="softmax",
             renorm=False, bias=False, scale=1.0),
        # the tiny float32 layer with a token per rank
        dict(name="ffn_tiny", op="ffn", bits=16, type="f32", R=4, S=1, E=16, K=2, H=128, Hp=256),
        # a ragged batch of 15 tokens at widths that no vector divides
        dict(name="ffn_odd", op="ffn", bits=16, type="bf16", R=3, S=5, E=21, K=4, H=1413, Hp=759),
        # decoding one sequence through a large layer
        dict(name="ffn_large_one", op="ffn", bits=16, type="bf16", R=1, S=1, E=256, K=8, H=7168, Hp=2048),
        # a decoding batch of 32 sequences, which reaches most of the experts
        dict(name="ffn_large_batch", op="ffn", bits=16, type="bf16", R=8, S=4, E=256, K=8, H=7168, Hp=2048),
        # decoding 8 sequences through the mid layer, weights in 4 bits
        dict(name="ffn4_mid_decode", op="ffn", bits=4, G=32, type="bf16", R=8, S=1, E=64, K=6, H=2048, Hp=1408),
        # a decoding batch of 16 sequences through the large layer, weights in 4 bits
        dict(name="ffn4_large_batch", op="ffn", bits=4, G=32, type="bf16", R=8, S=2, E=256, K=8, H=7168, Hp=2048),
        # one matrix in 4 bits and one token
        dict(name="project4_one", op="project", bits=4, G=128, type="bf16", R=1, S=1, E=1, K=1, H=7168, Hp=2048),
        # float32 rows at odd widths, a group size that the input width is no multiple of
        dict(name="project4_odd", op="project", bits=4, G=64, type="f32", R=4, S=3, E=16, K=3, H=1413, Hp=1531),
        # the mid layer's down projections into 4 bits and back, once a model is loaded
        dict(name="weights_mid", op="weights", G=32, type="bf16", E=64, H=1408, Hp=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, hi):
    width = _log(rng, 64, hi)
    # most models' widths are multiples of 64; the others are odd sizes
    return max(64, width // 64 * 64) if rng.random() < 0.6 else width


def draw(rng):
    op = rng.choice(["route", "route", "ffn", "ffn", "ffn", "project", "project", "weights"])
    R = rng.choice([1, 2, 4, 8])
    if op == "route":
        E = R * rng.randint(1, 384 // R)
        return dict(op=op, part=rng.choice(["forward", "backward"]), R=R, S=_log(rng, 1, 4096), E=E,
                    K=rng.randint(1, min(8, E)), score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                    bias=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    H, Hp, type_, G = _width(rng, 7168), _width(rng, 2048), rng.choice(["bf16", "bf16", "f32"]), rng.choice([32, 64, 128])
    E = R * _log(rng, 1, 256 // R)
    if op == "weights":
        return dict(op=op, G=G, type=type_, E=min(E, 64), H=H, Hp=Hp)
    case = dict(op=op, bits=16, type=type_, R=R, S=_log(rng, 1, 32 // R), E=E, K=rng.randint(1, min(8, E)), H=H, Hp=Hp)
    if rng.random() < 0.5:
        case.update(bits=4, G=G)
        case["S"] = min(case["S"], max(1, 16 // R))
    elif type_ == "f32":  # as many weight bytes as in bfloat16
        case["Hp"] = max(1, Hp // 2)
    return case


def work(case):
    if case["op"] == "route":
        T = case["R"] * case["S"]
        E, K = case["E"], case["K"]
        if case["part"] == "forward":
            return {"bytes": T * (4 * E + 8 * K) + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
        scores = E if case["score"] == "softmax" and not case["renorm"] else K
        return {"bytes": T * (4 * E + 4 * scores + 8 * K), "flops": 8 * T * E}
    eb = 2 if case["type"] == "bf16" else 4
    n = case["H"] * case["Hp"]
    if case["op"] == "weights":
        kept = case["E"] * n * (0.5 + 2 / case["G"])
        return {"bytes": case["E"] * n * (eb + 4) + 2 * kept, "flops": 4 * case["E"] * n}
    T, E, K, H, Hp = (case["R"] * case["S"],) + tuple(case[k] for k in "E K H Hp".split())
    reached = E * (1 - (1 - K / E) ** T)  # experts that T tokens choose between them, all being as likely
    per = 0.5 + 2 / case["G"] if case["bits"] == 4 else eb
    matrices, wide = (3, H) if case["op"] == "ffn" else (1, Hp)
    return {"bytes": reached * matrices * n * per + T * (H * eb + 8 * K + 4 * wide),
            "flops": 2 * matrices * n * T * K}


# ------------------------------------------------------------------ inputs

def _logits(g, T, E, dev):
    """Router scores of tokens that prefer some experts to others."""
    return torch.randn(T, E, generator=g, device=dev).add_(0.5 * torch.randn(E, generator=g, device=dev))


def _normal(g, shape, std, t, dev):
    return torch.empty(shape, dtype=t, device=dev).normal_(0, std, generator=g)


def _codes(g, E, H, N, G, dev):
    """Weights in 4 bits: random codes, and scales as of normal values with a deviation of 1 / sqrt(H)."""
    words = torch.randint(-2 ** 31, 2 ** 31, (E, -(-H // 8), N), generator=g, dtype=torch.int32, device=dev)
    scales = (0.3 + 0.1 * torch.rand(E, -(-H // G), N, generator=g, device=dev)) / math.sqrt(H)
    return words, scales.to(torch.bfloat16)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)
    s = dict(case=case)
    f32, i32 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.int32, device=dev)
    if case["op"] == "weights":
        E, H, Hp, G = (case[k] for k in ("E", "H", "Hp", "G"))
        s["W"] = _normal(g, (E, H, Hp), 1 / math.sqrt(H), TYPES[case["type"]], dev)
        s["codes"] = torch.empty(E, -(-H // 8), Hp, **i32)
        s["scales"] = torch.empty(E, -(-H // G), Hp, dtype=torch.bfloat16, device=dev)
        s["values"] = torch.empty(E, H, Hp, **f32)
        return s
    R, S, E, K = (case[k] for k in "RSEK")
    T = R * S
    logits = _logits(g, T, E, dev)
    chosen = torch.topk(logits, K).indices
    if case["op"] == "route":
        s["logits"] = logits.view(R, S, E)
        if case["part"] == "forward":
            # what balances the loads: less for the experts that are preferred, and equal steps, so that some tie
            s["bias"] = 0.001 * torch.randint(-50, 51, (E,), generator=g, device=dev).float() if case["bias"] else None
            s["topk_idx"], s["gates"] = torch.empty(R, S, K, **i32), torch.empty(R, S, K, **f32)
        else:
            s["topk_idx"] = chosen.to(torch.int32).view(R, S, K)
            s["dgates"] = torch.randn(R, S, K, generator=g, **f32)
            s["dlogits"] = torch.empty(R, S, E, **f32)
        return s
    t, H, Hp = TYPES[case["type"]], case["H"], case["Hp"]
    s["X"] = torch.randn(R, S, H, generator=g, **f32).to(t)
    s["topk_idx"] = chosen.to(torch.int32).view(R, S, K)
    s["gates"] = torch.softmax(logits.gather(1, chosen), -1).view(R, S, K)
    shapes = {"gu": (H, 2 * Hp), "down": (Hp, H)} if case["op"] == "ffn" else {"w": (H, Hp)}
    for name, (rows, cols) in shapes.items():
        if case["bits"] == 4:
            s[name] = _codes(g, E, rows, cols, case["G"], dev)
        else:
            s[name] = _normal(g, (E, rows, cols), 1 / math.sqrt(rows), t, dev)
    s["out"] = torch.empty(R, S, H if case["op"] == "ffn" else Hp, **f32)
    return s


# ------------------------------------------------------------------ plain forms

def _scores(l, score):
    """Router scores of float32 logits; what is masked (NaN, -inf) scores 0."""
    off = ~(l > -math.inf)
    l = l.clamp(max=LARGEST)
    if score == "sigmoid":
        return (1 / (1 + torch.exp(-l))).masked_fill(off, 0)
    p = torch.exp(l - l.masked_fill(off, -math.inf).amax(-1, keepdim=True)).masked_fill(off, 0)
    return p / p.sum(-1, keepdim=True)


def _route(s):
    case = s["case"]
    E, K, scale = case["E"], case["K"], case["scale"]
    l = s["logits"].view(-1, E)
    if case["part"] == "forward":
        # scores differ by less than 32 bits hold where experts are chosen: they are compared in 64
        key = l if s["bias"] is None else _scores(l.double(), case["score"]) + s["bias"].double()
        ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :K]
        w = _scores(l, case["score"]).gather(1, ids)
        gates = scale * (w / w.sum(-1, keepdim=True) if case["renorm"] else w)
        return {"topk_idx": ids.to(torch.int32).view(s["topk_idx"].shape), "gates": gates.view(s["gates"].shape)}
    ids = s["topk_idx"].view(-1, K).long()
    p = _scores(l, case["score"])
    w, c = p.gather(1, ids), scale * s["dgates"].view(-1, K)
    if case["renorm"]:
        q = w / w.sum(-1, keepdim=True)
        dw = q * (c - (q * c).sum(-1, keepdim=True))
        dl = torch.zeros_like(l).scatter_(1, ids, dw if case["score"] == "softmax" else dw * (1 - w))
    elif case["score"] == "softmax":
        dl = p * (torch.zeros_like(l).scatter_(1, ids, c) - (w * c).sum(-1, keepdim=True))
    else:
        dl = torch.zeros_like(l).scatter_(1, ids, c * w * (1 - w))
    return {"dlogits": dl.view(s["logits"].shape)}


def _shifts(device):
    i = torch.arange(8, device=device)
    return (4 * (i // 2) + 16 * (i % 2)).to(torch.int32).view(1, 1, 8, 1)


def _values4(words, scales, H, G):
    """The float32 values of 4-bit weights [n, H, N]."""
    n, J, N = words.shape
    q = ((words.unsqueeze(2) >> _shifts(words.device)) & 15).float() - 8
    return q.view(n, 8 * J, N)[:, :H] * scales.float().repeat_interleave(G, 1)[:, :H]


def _save4(w, G):
    """Words [E, ceil(H/8), N] and scales [E, ceil(H/G), N] of float32 weights."""
    E, H, N = w.shape
    groups = -(-H // G)
    wide = torch.nn.functional.pad(w, (0, 0, 0, groups * G - H)).view(E, groups, G, N)
    scales = (wide.abs().amax(2) / 7).to(torch.bfloat16)
    q = (wide / scales.float().unsqueeze(2)).round().clamp(-8, 7).nan_to_num(0).view(E, -1, N)
    q = (q[:, :-(-H // 8) * 8].reshape(E, -1, 8, N).to(torch.int32) + 8) << _shifts(w.device)
    return q.sum(2).to(torch.int32), scales


def _weights_of_pairs(s, name, rows):
    """The weight matrix of every pair of a token and an expert, in float32."""
    case, ids = s["case"], s["topk_idx"].view(-1).long()
    if case["bits"] == 4:
        words, scales = s[name]
        return _values4(words[ids], scales[ids], rows, case["G"])
    return s[name][ids].float()


def _experts(s):
    case = s["case"]
    K, H, Hp = case["K"], case["H"], case["Hp"]
    x = s["X"].float().view(-1, 1, H).repeat_interleave(K, 0)
    if case["op"] == "ffn":
        y = torch.bmm(x, _weights_of_pairs(s, "gu", H))
        gate, up = y[..., :Hp], y[..., Hp:]
        y = torch.bmm(gate / (1 + torch.exp(-gate)) * up, _weights_of_pairs(s, "down", Hp))
    else:
        y = torch.bmm(x, _weights_of_pairs(s, "w", H))
    return {"out": (y.view(-1, K, y.shape[-1]) * s["gates"].view(-1, K, 1)).sum(1).view(s["out"].shape)}


def _plain(s):
    case = s["case"]
    if case["op"] == "route":
        return _route(s)
    if case["op"] == "weights":
        return {"values": _values4(*_save4(s["W"].float(), case["G"]), case["H"], case["G"])}
    return _experts(s)


# ------------------------------------------------------------------ the library's calls

def _library(s):
    import load_balanced_dispatch_amd as m
    case = s["case"]
    if case["op"] == "weights":
        shape = tuple(case[k] for k in ("E", "H", "Hp", "G"))
        m.moonep_save4(*shape, s["W"], s["codes"], s["scales"])
        m.moonep_load4(*shape, s["codes"], s["scales"], s["values"])
        return {"values": s["values"]}
    d = m.make_dims(case["R"], case["E"], 0, case["S"], case["K"])
    if case["op"] == "route":
        how = (d, case["score"], case["renorm"], case["scale"], s["logits"])
        if case["part"] == "forward":
            m.moonep_route(*how, s["bias"], s["topk_idx"], s["gates"])
            return {"topk_idx": s["topk_idx"], "gates": s["gates"]}
        m.moonep_route_backward(*how, s["topk_idx"], s["dgates"], s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if "workspace" not in s:  # a program keeps it next to its buffers
        nbytes = m.moonep_few_workspace_bytes(d, case["H"], case["Hp"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    size, rows = (d, case["H"], case["Hp"]), (s["X"], s["topk_idx"], s["gates"])
    if case["bits"] == 4:
        size += (case["G"],)
        if case["op"] == "ffn":
            m.moonep_few_ffn4(*size, *rows, *s["gu"], *s["down"], s["out"], s["workspace"])
        else:
            m.moonep_few_layer4(*size, *rows, *s["w"], s["out"], s["workspace"])
    elif case["op"] == "ffn":
        m.moonep_few_ffn(*size, *rows, s["gu"], s["down"], s["out"], s["workspace"])
    else:
        m.moonep_few_layer(*size, *rows, s["w"], s["out"], s["workspace"])
    return {"out": s["out"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits

def _matrix64(s, name, e, rows):
    """The weight matrix of expert e in float64."""
    if s["case"]["bits"] != 4:
        return s[name][e].double()
    words, scales = s[name][0][e].long(), s[name][1][e].double()
    w = torch.empty(words.shape[0] * 8, words.shape[1], dtype=torch.float64, device=words.device)
    for i in range(8):
        w[i::8] = ((words >> (4 * (i // 2) + 16 * (i % 2))) % 16 - 8).double()
    G = s["case"]["G"]
    for first in range(0, rows, G):
        w[first:first + G] *= scales[first // G]
    return w[:rows]


def _route64(s):
    case = s["case"]
    E, K = case["E"], case["K"]
    l = s["logits"].reshape(-1, E).double()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    token = torch.arange(l.shape[0], device=l.device)[:, None]
    if case["part"] == "forward":
        key = l.clone() if s["bias"] is None else score + s["bias"].double()
        ids = []
        for _ in range(K):  # the largest that is left, the first of equals
            best = torch.where(key == key.amax(1, keepdim=True), torch.arange(E, device=l.device), E).amin(1)
            ids.append(best)
            key[token[:, 0], best] = -math.inf
        ids = torch.stack(ids, 1)
        picked = score[token, ids]
        if case["renorm"]:
            picked = picked / picked.sum(1, keepdim=True)
        return {"topk_idx": ids.to(torch.int32).view(s["topk_idx"].shape),
                "gates": (case["scale"] * picked).view(s["gates"].shape)}
    ids = s["topk_idx"].reshape(-1, K).long()
    up = case["scale"] * s["dgates"].reshape(-1, K).double()
    picked = score[token, ids]
    if case["renorm"]:
        total = picked.sum(1, keepdim=True)
        up = (up - (up * picked).sum(1, keepdim=True) / total) / total
    dscore = torch.zeros_like(l)
    dscore[token, ids] = up
    if case["score"] == "sigmoid":
        dl = dscore * score * (1 - score)
    else:
        dl = score * (dscore - (dscore * score).sum(1, keepdim=True))
    return {"dlogits": dl.view(s["logits"].shape)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route64(s)
    if case["op"] == "weights":
        E, H, Hp, G = (case[k] for k in ("E", "H", "Hp", "G"))
        values = s["W"].double()
        for first in range(0, H, G):
            w = values[:, first:first + G]
            # the scale is held in 16 bits, of a quotient in 32
            scale = (w.abs().amax(1, keepdim=True).float() / 7).to(torch.bfloat16).double()
            w.copy_(torch.clamp(torch.round(w / scale), -8, 7) * scale)
        return {"values": values}
    K, H, Hp = case["K"], case["H"], case["Hp"]
    x, ids, gates = s["X"].double().view(-1, H), s["topk_idx"].view(-1, K), s["gates"].double().view(-1, K)
    out = torch.zeros(x.shape[0], s["out"].shape[-1], dtype=torch.float64, device=x.device)
    for e in ids.unique().tolist():
        token, k = (ids == e).nonzero(as_tuple=True)
        if case["op"] == "ffn":
            y = x[token] @ _matrix64(s, "gu", e, H)
            y = (y[:, :Hp] * torch.sigmoid(y[:, :Hp]) * y[:, Hp:]) @ _matrix64(s, "down", e, Hp)
        else:
            y = x[token] @ _matrix64(s, "w", e, H)
        out.index_add_(0, token, y * gates[token, k][:, None])
    return {"out": out.view(s["out"].shape)}
