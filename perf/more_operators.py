"""The 8-bit floating point path and the tokens of a layer of experts as measured cases: the quantiser to blocks of
128 values with a scale each, the projection of such rows by such weights, the same by the experts of each row, and
the tokens sorted by expert and back, with their gradients.

Each case is one operator at one size.  ``run`` computes it either in plain torch operations (32-bit arithmetic, one
rounding at the end) or, where ``own`` is true, with this library's entry points; ``exact`` computes it in 64 bits,
from the definition:

  quant    v = x, silu(gate) * x, or x[rows];  of each block of 128 values of a row, or of 128 x 128 of a weight:
           scale = max|v| / 448,  q = e4m3(v * 448 / max|v|)
  linear   y[m, n] = sum_b x_scale[m, b] w_scale[n / 128, b] sum_(k in block b) x[m, k] W[n, k]  (+ residual[m, n])
  experts  the same for rows sorted by expert, each by its expert's weight; rows of no expert stay as they were
  tokens   (token, choice) sorted by expert, in order within one:  rows[p] the token of sorted row p, pos[t, j] the
           sorted row of a choice, -1 where the choice is no expert;   gathered[p] = x[rows[p]];
           out[t] = residual[t] + sum_j weight[t, j] y[pos[t, j]]
           and their gradients:  grad_y[pos[t, j]] = weight[t, j] grad_out[t],  grad_weight[t, j] = <grad_out[t],
           y[pos[t, j]]>,  grad_x[t] = sum_j grad_gathered[pos[t, j]]
"""
from __future__ import annotations

import math

import torch

own = False

F8 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # a decode batch of 64 tokens entering a layer of 384 experts, 8 of which each token takes: sorted and quantised
        {"name": "quant rows t64", "op": "quant", "M": 64, "K": 7168, "form": "rows", "k": 8},
        # the gated activation of a long prompt
        {"name": "quant gate m4096", "op": "quant", "M": 4096, "K": 16384, "form": "gate", "k": 0},
        # a weight with ragged sizes as it is loaded: the last blocks of both directions are short
        {"name": "quant weight odd", "op": "quant", "M": 5001, "K": 4112, "form": "weight", "k": 0},
        # one token through the wide input projection
        {"name": "linear m1 wide", "op": "linear", "M": 1, "N": 12288, "K": 7168, "epilogue": "bf16"},
        # the largest decode batch through the deep-K output projection, residual added
        {"name": "linear m64 deep", "op": "linear", "M": 64, "N": 7168, "K": 16384, "epilogue": "bf16_residual"},
        # a short prompt with ragged sizes, scores kept in fp32
        {"name": "linear m333 odd", "op": "linear", "M": 333, "N": 5001, "K": 4112, "epilogue": "fp32"},
        # a long prompt through the wide input projection
        {"name": "linear m4096 wide", "op": "linear", "M": 4096, "N": 12288, "K": 7168, "epilogue": "bf16"},
        # one token's 8 experts of 64, small ones: latency alone
        {"name": "experts t1", "op": "experts", "T": 1, "k": 8, "E": 64, "N": 1024, "K": 1024, "dropped": 0.0},
        # a decode batch: the experts' weights from HBM, a row or two for each of them
        {"name": "experts t16", "op": "experts", "T": 16, "k": 8, "E": 384, "N": 2048, "K": 4096, "dropped": 0.0},
        # a prompt, popular experts among them, some choices dropped
        {"name": "experts t2048", "op": "experts", "T": 2048, "k": 8, "E": 32, "N": 4096, "K": 4096, "dropped": 0.02},
        # a decode batch of 16 tokens to its experts and back
        {"name": "tokens t16", "op": "tokens", "T": 16, "k": 8, "E": 384, "K": 7168, "dropped": 0.0, "train": False},
        # a training batch, forward and backward, some choices dropped
        {"name": "tokens t4096 train", "op": "tokens", "T": 4096, "k": 8, "E": 384, "K": 7168, "dropped": 0.02, "train": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "experts", "experts", "tokens"])
    if op == "quant":
        form = rng.choice(["plain", "gate", "rows", "weight"])
        k = rng.choice([1, 2, 4, 6, 8]) if form == "rows" else 0
        return {"op": op, "M": _log(rng, 1, 4096 // max(1, k)), "K": _log(rng, 128, 16384), "form": form, "k": k}
    if op == "linear":
        N, K = _log(rng, 64, 16384), 16 * _log(rng, 16, 1024)
        M = _log(rng, 1, max(1, min(4096, 4096 * 12288 * 7168 // (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "epilogue": rng.choice(["bf16", "bf16_residual", "fp32"])}
    dropped = rng.choice([0.0, 0.0, 0.02, 0.3])
    if op == "experts":
        E, k = _log(rng, 8, 384), rng.choice([1, 2, 4, 6, 8])
        N, K = _log(rng, 256, 4096), 16 * _log(rng, 16, 256)
        return {"op": op, "T": _log(rng, 1, 2048), "k": k, "E": min(E, max(8, (3 << 30) // (N * K))), "N": N, "K": K,
                "dropped": dropped}
    return {"op": op, "T": _log(rng, 1, 4096), "k": rng.choice([1, 2, 4, 6, 8]), "E": _log(rng, 8, 384),
            "K": _log(rng, 256, 7168), "dropped": dropped, "train": rng.random() < 0.5}


def _blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------------------------ inputs
def _choices(case, g):
    """Each token's k best of E scores, some experts popular; -1 where a choice was beyond its expert's capacity."""
    T, k, E = case["T"], case["k"], case["E"]
    scores = torch.randn(T, E, generator=g, device=g.device) + 0.5 * torch.randn(E, generator=g, device=g.device)
    chosen = torch.topk(scores, k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        chosen[torch.rand(T, k, generator=g, device=g.device) < case["dropped"]] = -1
    return chosen


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) * std).to(dtype)

    def eights(*shape):           # quantised normal rows: the largest of 128 is about 2.7 sigma = 448
        return normal(*shape).mul_(160.0).clamp_(-448.0, 448.0).to(F8)

    def positive(*shape, mean):
        return mean * (0.5 + torch.rand(*shape, generator=g, device="cuda"))

    s = dict(case)
    if case["op"] == "quant":
        M, K = case["M"], case["K"]
        if case["form"] == "gate":     # one [M, 2K] output of a fused gate/up projection: both halves are views of it
            both = normal(M, 2 * K, std=1.5)
            s["gate"], s["x"] = both[:, :K], both[:, K:]
        else:
            s["gate"], s["x"] = None, normal(M, K, std=0.02 if case["form"] == "weight" else 1.5)
        s["rows"] = None
        if case["form"] == "rows":     # every token k times, in the order of the experts they go to
            s["rows"] = torch.randperm(M * case["k"], generator=g, device="cuda").div(case["k"], rounding_mode="floor").int()
    elif case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["x_scale"] = eights(M, K), positive(M, _blocks(K), mean=1 / 160)
        s["W"], s["w_scale"] = eights(N, K), positive(_blocks(N), _blocks(K), mean=1 / (160 * math.sqrt(K)))
        s["residual"] = normal(M, N) if case["epilogue"] == "bf16_residual" else None
    elif case["op"] == "experts":
        T, k, E, N, K = (case[c] for c in ("T", "k", "E", "N", "K"))
        chosen = _choices(case, g).flatten()
        counts = torch.bincount(chosen[chosen >= 0], minlength=E)
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["x"], s["x_scale"] = eights(T * k, K), positive(T * k, _blocks(K), mean=1 / 160)
        s["W"] = eights(E, N, K)
        s["w_scale"] = positive(E, _blocks(N), _blocks(K), mean=1 / (160 * math.sqrt(K)))
    else:
        T, k, E, K = (case[c] for c in ("T", "k", "E", "K"))
        s["expert"] = _choices(case, g)
        s["weight"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1)
        s["x"], s["residual"], s["y"] = normal(T, K), normal(T, K), normal(T * k, K)
        if case["train"]:
            s["grad_out"], s["grad_gathered"] = normal(T, K), normal(T * k, K)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:      # the plan and the buffers that a program keeps
        from projection_gemm_gb300 import skg

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        if case["op"] == "quant":
            M, K = case["M"] * max(1, case["k"]), case["K"]
            s["q"] = empty(M, K, dtype=F8)
            s["scale"] = empty(_blocks(M) if case["form"] == "weight" else M, _blocks(K), dtype=torch.float32)
        elif case["op"] == "linear":
            s["plan"] = skg.F8Plan(case["M"], case["N"], case["K"], case["epilogue"], static_weights=True)
            s["out"] = empty(case["M"], case["N"], dtype=torch.float32 if case["epilogue"] == "fp32" else torch.bfloat16)
        elif case["op"] == "experts":
            rows = case["T"] * case["k"]
            s["plan"] = skg.F8Plan(rows, case["N"], case["K"], "bf16", experts=case["E"], static_weights=True)
            s["out"] = torch.zeros(rows, case["N"], dtype=torch.bfloat16, device="cuda")
        else:
            T, k, K = case["T"], case["k"], case["K"]
            s["offsets"] = empty(case["E"] + 1, dtype=torch.int32)
            s["rows"], s["pos"] = empty(T * k, dtype=torch.int32), empty(T, k, dtype=torch.int32)
            s["gathered"], s["out"] = empty(T * k, K), empty(T, K)
            if case["train"]:
                s["grad_y"] = torch.zeros(T * k, K, dtype=torch.bfloat16, device="cuda")
                s["grad_weight"], s["grad_x"] = empty(T, k, dtype=torch.float32), empty(T, K)
    return s


# ------------------------------------------------------------------------------------------- plain form
def _dequantised(q, scale, rows_a_block):
    """The values that q stands for, in fp32: a scale for rows_a_block x 128 of them."""
    s = scale.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]
    if rows_a_block > 1:
        s = s.repeat_interleave(rows_a_block, dim=-2)[..., :q.shape[-2], :]
    return q.float() * s


def _quantised(v, rows_a_block):
    M, K = v.shape
    b, rb = _blocks(K), -(-M // rows_a_block)
    padded = torch.nn.functional.pad(v, (0, b * BLOCK - K, 0, rb * rows_a_block - M)).view(rb, rows_a_block, b, BLOCK)
    largest = padded.abs().amax(dim=(1, 3), keepdim=True)
    q = padded * torch.where(largest > 0, 448.0 / largest, 0.0)
    return q.view(rb * rows_a_block, b * BLOCK)[:M, :K].to(F8), (largest / 448.0).view(rb, b)


def _plain_tokens(s):
    T, k, E = s["T"], s["k"], s["E"]
    flat = s["expert"].flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device="cuda").index_add_(0, key, torch.ones_like(key))
    bounds = counts.cumsum(0)[:E]
    offsets = torch.cat([torch.zeros_like(bounds[:1]), bounds]).to(torch.int32)
    here = key[order] < E
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    pos = torch.where(key < E, place, -1).view(T, k)
    rows = torch.where(here, order // k, -1)
    answer = {"offsets": offsets, "rows": rows.to(torch.int32), "pos": pos.to(torch.int32),
              "gathered": torch.where(here[:, None], s["x"][rows.clamp(min=0)], 0.0)}
    taken = pos >= 0
    out = s["residual"].float()
    for j in range(k):
        out = out + torch.where(taken[:, j, None], s["y"][pos[:, j].clamp(min=0)].float() * s["weight"][:, j, None], 0.0)
    answer["out"] = out.to(torch.bfloat16)
    if s["train"]:
        grad = s["grad_out"].float()
        grad_y, grad_weight = torch.zeros_like(s["y"]), torch.zeros(T, k, device="cuda")
        grad_x = torch.zeros_like(grad)
        for j in range(k):
            t, p = taken[:, j].nonzero()[:, 0], pos[taken[:, j], j]
            grad_y[p] = (grad[t] * s["weight"][t, j, None]).to(torch.bfloat16)
            grad_weight[t, j] = (grad[t] * s["y"][p].float()).sum(1)
            grad_x[t] += s["grad_gathered"][p].float()
        answer.update(grad_y=grad_y, grad_weight=grad_weight, grad_x=grad_x.to(torch.bfloat16))
    return answer


def _plain(s):
    if s["op"] == "quant":
        v = s["x"].float()
        if s["gate"] is not None:
            g = s["gate"].float()
            v = g / (1.0 + torch.exp(-g)) * v
        if s["rows"] is not None:
            v = v[s["rows"].long()]
        q, scale = _quantised(v, BLOCK if s["form"] == "weight" else 1)
        return {"q": q, "scale": scale}
    if s["op"] == "tokens":
        return _plain_tokens(s)
    x = _dequantised(s["x"], s["x_scale"], 1)
    if s["op"] == "linear":
        y = x @ _dequantised(s["W"], s["w_scale"], BLOCK).t()
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y if s["epilogue"] == "fp32" else y.to(torch.bfloat16)}
    y = torch.zeros(x.shape[0], s["N"], dtype=torch.bfloat16, device="cuda")
    bounds = s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            y[a:b] = (x[a:b] @ _dequantised(s["W"][e], s["w_scale"][e], BLOCK).t()).to(torch.bfloat16)
    return {"y": y}


# ------------------------------------------------------------------------------------ this library's form
def _own(s):
    from projection_gemm_gb300 import skg
    if s["op"] == "quant":
        if s["form"] == "weight":
            skg.skg_quantize_f8_weights(s["x"], s["q"], s["scale"])
        else:
            skg.skg_quantize_f8(s["x"], s["gate"], s["q"], s["scale"], rows=s["rows"])
        return {"q": s["q"], "scale": s["scale"]}
    if s["op"] == "linear":
        s["plan"].run(s["x"], s["x_scale"], s["W"], s["w_scale"], s["residual"], s["out"])
        return {"y": s["out"]}
    if s["op"] == "experts":
        s["plan"].run(s["x"], s["x_scale"], s["W"], s["w_scale"], None, s["out"], offsets=s["offsets"])
        return {"y": s["out"]}
    skg.skg_experts_sort(s["expert"], s["offsets"], s["rows"], s["pos"])
    skg.skg_experts_gather(s["x"], s["rows"], s["gathered"])
    skg.skg_experts_combine(s["y"], s["pos"], s["weight"], s["residual"], s["out"])
    names = ["offsets", "rows", "pos", "gathered", "out"]
    if s["train"]:
        skg.skg_experts_combine_grad(s["grad_out"], s["y"], s["pos"], s["weight"], s["grad_y"], s["grad_weight"])
        skg.skg_experts_combine(s["grad_gathered"], s["pos"], None, None, s["grad_x"])
        names += ["grad_y", "grad_weight", "grad_x"]
    return {n: s[n] for n in names}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------------------- 64-bit values
def _exact_e4m3(v):
    """v to the nearest number of 4 significant bits, half to even; below 2^-6 to the nearest multiple of 2^-9."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_blocks(v, tall):
    q, scale = torch.empty_like(v), v.new_empty(-(-v.shape[0] // tall), _blocks(v.shape[1]))
    for b in range(scale.shape[1]):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        largest = part.abs().amax(1)
        largest = torch.stack([c.max() for c in largest.split(tall)]) if tall > 1 else largest
        scale[:, b] = largest / 448
        step = scale[:, b].repeat_interleave(tall)[:v.shape[0], None]
        q[:, b * BLOCK:(b + 1) * BLOCK] = _exact_e4m3(torch.nan_to_num(part / step))
    return q, scale


def _exact_product(x, x_scale, W, w_scale):
    x, W = x.double(), W.double()
    for b in range(_blocks(x.shape[1])):
        k = slice(b * BLOCK, (b + 1) * BLOCK)
        x[:, k] *= x_scale[:, b, None].double()
        for n in range(w_scale.shape[0]):
            W[n * BLOCK:(n + 1) * BLOCK, k] *= w_scale[n, b].double()
    return torch.mm(x, W.T)


def _exact_tokens(s):
    T, k, E = s["T"], s["k"], s["E"]
    chosen = s["expert"].flatten().tolist()
    lists = [[] for _ in range(E)]
    for i, e in enumerate(chosen):
        if 0 <= e < E:
            lists[e].append(i)
    order = [i for at in lists for i in at]
    offsets = [0]
    for at in lists:
        offsets.append(offsets[-1] + len(at))
    pos = [-1] * (T * k)
    for p, i in enumerate(order):
        pos[i] = p
    routed = torch.tensor(order, dtype=torch.long, device="cuda")
    token, n = routed // k, len(order)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    gathered = torch.zeros(T * k, s["K"], dtype=torch.float64, device="cuda")
    gathered[:n] = s["x"].double()[token]
    w = s["weight"].double().flatten()[routed, None]
    out = s["residual"].double().index_add(0, token, s["y"][:n].double() * w)
    answer = {"offsets": ints(offsets), "rows": ints([i // k for i in order] + [-1] * (T * k - n)),
              "pos": ints(pos).view(T, k), "gathered": gathered, "out": out}
    if s["train"]:
        grad = s["grad_out"].double()[token]
        grad_y, grad_weight = torch.zeros_like(gathered), torch.zeros(T * k, dtype=torch.float64, device="cuda")
        grad_y[:n] = grad * w
        grad_weight[routed] = torch.linalg.vecdot(grad, s["y"][:n].double())
        grad_x = torch.zeros_like(out).index_add(0, token, s["grad_gathered"][:n].double())
        answer.update(grad_y=grad_y, grad_weight=grad_weight.view(T, k), grad_x=grad_x)
    return answer


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quant":
        v = s["x"].double()
        if s["gate"] is not None:
            g = s["gate"].double()
            v = torch.sigmoid(g) * g * v
        if s["rows"] is not None:
            v = v.index_select(0, s["rows"])
        q, scale = _exact_blocks(v, BLOCK if case["form"] == "weight" else 1)
        return {"q": q, "scale": scale}
    if case["op"] == "tokens":
        return _exact_tokens(s)
    if case["op"] == "linear":
        y = _exact_product(s["x"], s["x_scale"], s["W"], s["w_scale"])
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    y = torch.zeros(case["T"] * case["k"], case["N"], dtype=torch.float64, device="cuda")
    bounds = s["offsets"].tolist()
    for e in range(case["E"]):
        at = slice(bounds[e], bounds[e + 1])
        if at.stop > at.start:
            y[at] = _exact_product(s["x"][at], s["x_scale"][at], s["W"][e], s["w_scale"][e])
    return {"y": y}


# ------------------------------------------------------------------------------------------------- work
def work(case):
    K = case["K"]
    if case["op"] == "quant":
        M, gated, k = case["M"], case["form"] == "gate", max(1, case["k"])
        scales = (_blocks(M) if case["form"] == "weight" else M * k) * _blocks(K)
        return {"bytes": 2 * (2 if gated else 1) * M * K + k * M * K + 4 * scales + (4 * M * k if case["k"] else 0),
                "flops": (8 if gated else 3) * M * k * K}
    if case["op"] == "linear":
        M, N = case["M"], case["N"]
        out = {"bf16": 2, "bf16_residual": 4, "fp32": 4}[case["epilogue"]]
        return {"bytes": N * K + M * K + 4 * _blocks(K) * (M + _blocks(N)) + out * M * N, "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    rows = max(1, round(T * k * (1 - case["dropped"])))
    if case["op"] == "experts":
        N = case["N"]
        chosen = _choices(case, torch.Generator().manual_seed(1))
        taken = len(torch.unique(chosen[chosen >= 0]))        # experts with a row: of other choices, about as many
        return {"bytes": int(taken * (N * K + 4 * _blocks(N) * _blocks(K)) + rows * (K + 4 * _blocks(K) + 2 * N) + 4 * E),
                "flops": 2 * rows * N * K}
    wide = 2 * K
    moved = T * wide + T * k * wide + rows * wide + 2 * T * wide                      # x, gathered; y, residual, out
    index = 4 * (3 * T * k + E) + 4 * T * k
    if not case["train"]:
        return {"bytes": moved + index, "flops": 2 * rows * K}
    moved += T * wide + 2 * rows * wide + rows * wide + T * wide      # grad_out, y, grad_y; grad_gathered, grad_x
    return {"bytes": moved + index + 8 * T * k, "flops": (2 + 3 + 1) * rows * K}
