"""The feed-forward operators, as they are timed: linear layers with bias,
activation and residual in the epilogue of the product, their backward pass,
and a whole mixture-of-experts layer for a few tokens.

    Y  = act(X W^T + b) + R          X: M x K, W: N x K, b: N, R and Y: M x N
    Z  = X W^T + b                   kept for the backward pass when training
    G  = dY * act'(Z)                dX = G W,  dW = G^T X,  db = sum of G's rows

    p  = softmax(X Wr^T) over E experts, the k largest of a token (ties: the
         lowest index), their weights w = p, or p over the sum of the k
    Y  = sum_j w_j W2[e_j] (act(W1[e_j] x))                     plain experts
    Y  = sum_j w_j W2[e_j] (act(Wg[e_j] x) * (Wu[e_j] x))       gated experts,
         W1[e] holding the F rows of Wg[e] and then the F rows of Wu[e]

`own` chooses between the elementary form and the library's operators.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu_erf", "gelu_tanh")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token through an attention output projection: latency and one
        # pass over a square weight
        dict(name="linear_row_bf16", op="linear", type="bf16", M=1, N=4096, K=4096, act="none",
             bias=True, residual=True, keep=False),
        # sixteen decoding sequences through the wide product of a feed-forward block
        dict(name="linear_decode16_bf16", op="linear", type="bf16", M=16, N=14336, K=4096,
             act="gelu_tanh", bias=True, residual=False, keep=False),
        # a ragged prefill whose rows start on 2-byte boundaries only
        dict(name="linear_ragged_f16", op="linear", type="f16", M=777, N=1000, K=1001, act="silu",
             bias=True, residual=True, keep=False),
        # the same block in fp32, with the residual stream added
        dict(name="linear_f32", op="linear", type="f32", M=2048, N=4096, K=4096, act="gelu_erf",
             bias=True, residual=True, keep=False),
        # a training step's forward pass: 8192 tokens, the sum kept for the backward pass
        dict(name="linear_train_bf16", op="linear", type="bf16", M=8192, N=14336, K=4096,
             act="gelu_tanh", bias=True, residual=False, keep=True),
        # the backward pass of a small fine-tuning batch on a wide layer
        dict(name="backward_few_bf16", op="backward", type="bf16", M=16, N=4096, K=4096,
             act="relu", bias=True),
        # a ragged batch through an odd-sized adapter layer
        dict(name="backward_ragged_f16", op="backward", type="f16", M=515, N=1000, K=776,
             act="silu", bias=True),
        # the backward pass of a training step's wide layer
        dict(name="backward_train_bf16", op="backward", type="bf16", M=4096, N=14336, K=4096,
             act="gelu_tanh", bias=True),
        # one decoding sequence, many small experts: latency
        dict(name="moe_1_bf16", op="moe", type="bf16", T=1, D=2048, F=1024, E=64, k=8, act="silu",
             gated=True, renorm=True),
        # odd sizes in fp32, plain experts
        dict(name="moe_5_f32", op="moe", type="f32", T=5, D=515, F=333, E=9, k=3, act="gelu_erf",
             gated=False, renorm=False),
        # sixteen sequences, few large experts
        dict(name="moe_16_f16", op="moe", type="f16", T=16, D=4096, F=14336, E=8, k=2,
             act="gelu_tanh", gated=True, renorm=True),
        # sixty-four sequences, nearly every one of many experts in use
        dict(name="moe_64_bf16", op="moe", type="bf16", T=64, D=2048, F=768, E=128, k=8,
             act="silu", gated=True, renorm=True),
    ]


def _size(rng, lo, hi):
    """A size of [lo, hi], even over the logarithm; half of them multiples of
    8 (where that stays in the range), the others as they fall, odd ones too."""
    v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    if rng.random() < 0.5 and v >= 8:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    t = rng.choice(("bf16", "bf16", "f16", "f32"))
    act = rng.choice(ACTS)
    op = rng.choice(("linear", "linear", "backward", "moe"))
    if op == "moe":
        while True:
            E = rng.choice((4, 8, 9, 16, 32, 60, 64, 128))
            c = dict(op="moe", type=t, T=_size(rng, 1, 64), D=_size(rng, 64, 4096),
                     F=_size(rng, 64, 14336), E=E, k=rng.randint(1, min(8, E)), act=act,
                     gated=rng.random() < 0.7, renorm=rng.random() < 0.5)
            if E * c["D"] * c["F"] * (3 if c["gated"] else 2) * SIZE[t] <= 2 << 30:
                return c
    most = 4e10 if t == "f32" else 4e11
    while True:
        c = dict(op=op, type=t, M=_size(rng, 1, 8192), N=_size(rng, 64, 14336),
                 K=_size(rng, 64, 14336), act=act, bias=rng.random() < 0.7)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, keep=rng.random() < 0.3)
        if (2 if op == "linear" else 4) * c["M"] * c["N"] * c["K"] <= most:
            return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt).mul_(std)

    s = dict(case=case)
    if case["op"] == "moe":
        T, D, F, E = case["T"], case["D"], case["F"], case["E"]
        s["X"] = normal(T, D)
        # router logits of standard deviation 1.5: a few experts stand out
        s["Wr"] = normal(E, D, std=1.5 / math.sqrt(D))
        s["W1"] = normal(E, 2 * F if case["gated"] else F, D, std=1 / math.sqrt(D))
        s["W2"] = normal(E, D, F, std=1 / math.sqrt(F))
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["X"] = normal(M, K)
        s["W"] = normal(N, K, std=1 / math.sqrt(K))
        if case["op"] == "linear":
            s["b"] = normal(N, std=0.5) if case["bias"] else None
            s["R"] = normal(M, N) if case["residual"] else None
        else:
            s["Z"] = normal(M, N) if case["act"] != "none" else None
            s["dY"] = normal(M, N, std=0.1)
    if own:
        import fp32_sgemm_02_amd as sg

        s["sg"] = sg
        s["act"] = (sg.ACT_NONE, sg.ACT_RELU, sg.ACT_SILU, sg.ACT_GELU_ERF,
                    sg.ACT_GELU_TANH)[ACTS.index(case["act"])]
    return s


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "linear":
        return _linear(s, c)
    if c["op"] == "backward":
        return _backward(s, c)
    return _moe(s, c)


def _run_own(s, c):
    sg = s["sg"]
    if c["op"] == "linear":
        return sg.linear(s["X"], s["W"], s["b"], act=s["act"], residual=s["R"],
                         keep_pre=c["keep"])
    if c["op"] == "backward":
        return sg.linear_backward(s["dY"], s["X"], s["W"], s["Z"], act=s["act"],
                                  need_bias=c["bias"])
    return sg.moe(s["X"], s["Wr"], s["W1"], s["W2"], c["k"], act=s["act"],
                  renormalize=c["renorm"], return_routing=True)


# ---- the elementary form, in 32 bits, rounded once at the end ----------------

def _act(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu_erf":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1 + torch.exp(-2 * u))
    return z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if name == "gelu_erf":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + \
            z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    q = 1 / (1 + torch.exp(-2 * u))
    return q + 2 * z * q * (1 - q) * du


def _linear(s, c):
    dt = s["X"].dtype
    z = s["X"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(c["act"], z)
    if s["R"] is not None:
        y = y + s["R"].float()
    return (y.to(dt), z.to(dt)) if c["keep"] else y.to(dt)


def _backward(s, c):
    dt = s["X"].dtype
    G = s["dY"].float()
    if s["Z"] is not None:
        G = G * _slope(c["act"], s["Z"].float())
    dX = G @ s["W"].float()
    dW = G.t() @ s["X"].float()
    return dX.to(dt), dW.to(dt), G.sum(0).to(dt) if c["bias"] else None


def _moe(s, c):
    X, W1, W2 = s["X"], s["W1"], s["W2"]
    T, k, E, F = c["T"], c["k"], c["E"], c["F"]
    # the logits in 64 bits: the k largest are chosen next to a border
    logits = X.double() @ s["Wr"].double().t()
    val, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    w = torch.exp(val - val[:, :1])
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    else:
        w = w / torch.exp(logits - val[:, :1]).sum(1, keepdim=True)
    w = w.float()
    x = X.float().t().contiguous()
    if T * k < E:
        # fewer choices than experts: gather each choice's expert
        pick = ids.reshape(-1)
        A, B = W1[pick].float(), W2[pick].float()
        h = A @ x.t().repeat_interleave(k, 0).unsqueeze(2)
        coef = w.reshape(-1, 1, 1)
    else:
        A, B = W1.float(), W2.float()
        h = A @ x
        table = torch.zeros(T, E, device=X.device).scatter(1, ids, w)
        coef = table.t().unsqueeze(1)
    h = _act(c["act"], h[:, :F]) * h[:, F:] if c["gated"] else _act(c["act"], h)
    y = B @ (h * coef)
    y = y.reshape(T, k, -1).sum(1) if T * k < E else y.sum(0).t()
    return y.to(X.dtype).contiguous(), ids.int(), w


# ---- the definition in 64 bits -----------------------------------------------

def _f(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu_erf":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def exact(case, seed):
    s = prepare(case, seed)
    name = case["act"]
    X = s["X"].double()
    if case["op"] == "linear":
        z = torch.matmul(X, s["W"].double().mT)
        if s["b"] is not None:
            z += s["b"].double()
        keep = z.clone() if case["keep"] else None
        y = _f(name, z)
        if s["R"] is not None:
            y = y + s["R"].double()
        return (y, keep) if case["keep"] else y
    if case["op"] == "backward":
        G = s["dY"].double()
        if s["Z"] is not None:
            z = s["Z"].double().requires_grad_()
            if name == "relu":   # the slope at 0 is taken as 0
                G = torch.where(z.detach() > 0, G, torch.zeros_like(G))
            else:
                with torch.enable_grad():
                    G, = torch.autograd.grad(_f(name, z), z, G)
        return (torch.matmul(G, s["W"].double()), torch.matmul(G.mT, X),
                torch.sum(G, 0) if case["bias"] else None)
    k, F = case["k"], case["F"]
    logits = torch.matmul(X, s["Wr"].double().mT)
    order = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    p = torch.softmax(logits, 1).gather(1, order)
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    Y = torch.zeros_like(X)
    for e in sorted(set(order.flatten().tolist())):
        rows, slot = (order == e).nonzero(as_tuple=True)
        h = torch.matmul(X[rows], s["W1"][e].double().mT)
        h = _f(name, h[:, :F]) * h[:, F:] if case["gated"] else _f(name, h)
        Y[rows] += p[rows, slot].unsqueeze(1) * torch.matmul(h, s["W2"][e].double().mT)
    return Y, order.int(), p


def work(case):
    z = SIZE[case["type"]]
    if case["op"] == "moe":
        T, D, F, E, k = (case[n] for n in ("T", "D", "F", "E", "k"))
        per = (3 if case["gated"] else 2) * D * F
        # experts that at least one token chooses, for choices spread evenly
        used = E * (1 - (1 - k / E) ** T)
        return dict(bytes=z * (used * per + E * D + 2 * T * D) + 8 * T * k,
                    flops=2 * T * (k * per + E * D))
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "linear":
        cells = M * N * (1 + int(case["residual"]) + int(case["keep"]))
        return dict(bytes=z * (M * K + N * K + cells + (N if case["bias"] else 0)),
                    flops=2 * M * N * K)
    cells = M * N * (1 + int(case["act"] != "none"))
    return dict(bytes=z * (2 * M * K + 2 * N * K + cells + (N if case["bias"] else 0)),
                flops=4 * M * N * K)
