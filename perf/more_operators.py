"""The products with what follows them in their epilogue: their cases, plain forms and 64-bit definitions.

Four uses are measured, all on BF16 operands:

  act       C = act(op(A) op(B) + bias) + R, C BF16 or FP32, R (the residual) and the bias
            optional; Z = op(A) op(B) + bias may be kept in BF16 for the backward pass. Gated:
            op(B) has 2 N columns, C = act(G) U with [G, U] = op(A) op(B) + bias, Z is [G, U].
  act_grad  the gradient of a layer's input taken on through the activation before it:
            D = op(A) op(B), dZ = D act'(Z), db the column sums of dZ. Gated, Z = [G, U]:
            dZ = [D U act'(G), D act(G)].
  ce        the softmax cross entropy of a head: z = X W^T over a vocabulary of V rows of W,
            lse_i = log sum_j exp z_ij, loss_i = lse_i - z_i[target_i]; a row whose target is
            not in 0 .. V - 1 is left out: its loss is 0.
  ce_grad   its gradients, given dloss and lse: dz_ij = dloss_i (exp(z_ij - lse_i) - [j = target_i]),
            0 in rows left out; dX = dz W, dW = dz^T X.

Activations:
  none  z             relu  max(z, 0)
  gelu  z Phi(z)      gelu_tanh  z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2
  silu  z / (1 + exp(-z))
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
ROOT_2_PI = math.sqrt(2.0 / math.pi)
IGNORED = -100


def _act(name, M, N, K, act, type="bf16", bias=False, residual="", keep_z=False, gated=False, trans_a=False, trans_b=True):
    return {"name": name, "op": "act", "M": M, "N": N, "K": K, "act": act, "type": type, "bias": bias,
            "residual": residual, "keep_z": keep_z, "gated": gated, "trans_a": trans_a, "trans_b": trans_b}


def _act_grad(name, M, N, K, act, gated=False):
    return {"name": name, "op": "act_grad", "M": M, "N": N, "K": K, "act": act, "gated": gated}


def _ce(name, op, T, V, D):
    return {"name": name, "op": op, "T": T, "V": V, "D": D}


def listed():
    return [
        # Decoding one token: the gate and up projections of an FFN and their gating in one call.
        _act("act_token", 1, 14336, 4096, "silu", gated=True),
        # 16 sequences decoding: the down projection, onto the residual stream.
        _act("act_down", 16, 4096, 14336, "none", bias=True, residual="bf16"),
        # Sizes that are whole tiles in no direction, rows off 16 bytes, an FP32 residual stream.
        _act("act_ragged", 3000, 5001, 1537, "gelu", "f32", bias=True, residual="f32", keep_z=True),
        # The FFN's up projection of 8192 tokens in training: Z is kept.
        _act("act_ffn", 8192, 14336, 4096, "gelu_tanh", bias=True, keep_z=True),
        # The gradient of its weights, dZ^T X, added to the FP32 sum of the micro-batches before.
        _act("act_weights", 14336, 4096, 8192, "none", "f32", residual="f32", trans_a=True, trans_b=False),
        # A small layer's backward pass.
        _act_grad("act_grad_small", 256, 1024, 1024, "relu"),
        # The gated FFN's backward pass on 8192 tokens: dY W_down, on to the gate's and up projection's outputs.
        _act_grad("act_grad_gated", 8192, 14336, 4096, "silu", gated=True),
        # The likelihood of one token: the vocabulary is read once.
        _ce("ce_token", "ce", 1, 32768, 1024),
        # Odd everywhere: rows of X and W off 16 bytes.
        _ce("ce_ragged", "ce", 1537, 50001, 1001),
        # The head of a training step on 8192 tokens.
        _ce("ce_train", "ce", 8192, 65536, 4096),
        # A small model's head, both gradients.
        _ce("ce_grad_small", "ce_grad", 64, 1000, 256),
        # The gradients of a training step's head, 4096 tokens.
        _ce("ce_grad_train", "ce_grad", 4096, 65536, 4096),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["act", "act", "act_grad", "ce", "ce_grad"])
    if op in ("ce", "ce_grad"):
        case = _ce("", op, size(1, 8192 if op == "ce" else 4096), size(128, 65536), size(64, 4096))
    else:
        M, N, K = size(1, 8192), size(64, 14336), size(64, 4096)
        if rng.random() < 0.3:
            N, K = K, N
        act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
        if op == "act_grad":
            case = _act_grad("", M, N, K, act, rng.random() < 0.4)
        elif rng.random() < 0.4:
            case = _act("", M, N, K, act, "bf16", rng.random() < 0.5, rng.choice(["", "bf16"]), rng.random() < 0.5, True,
                        trans_b=rng.random() < 0.7)
        else:
            kind = rng.choice(["f32", "bf16"])
            case = _act("", M, N, K, rng.choice(["none", act]), kind, rng.random() < 0.5, rng.choice(["", "bf16", "f32"]),
                        rng.random() < 0.3, False, rng.random() < 0.3, rng.random() < 0.7)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _normal(g, std, dtype, *size):
    return (torch.randn(size, generator=g, device="cuda") * std).to(dtype)


def _logits_lse(X, W):
    """log sum exp of X W^T's rows, FP32, some rows at a time."""
    w = W.float()
    return torch.cat([torch.logsumexp(x.float() @ w.t(), dim=1) for x in X.split(4096)])


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, bf16 = case["op"], torch.bfloat16
    if op in ("ce", "ce_grad"):
        T, V, D = case["T"], case["V"], case["D"]
        # Rows of W of length one, and of X part noise, part the target's row: the target's logit
        # is 8 or so among ones of spread 1, as a trained model's are. One row in ten is left out.
        W = _normal(g, D ** -0.5, bf16, V, D)
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        X = (torch.randn((T, D), generator=g, device="cuda") + 8.0 * W[target].float()).to(bf16)
        out = torch.rand((T,), generator=g, device="cuda") < 0.1
        target = torch.where(out, torch.full_like(target, IGNORED), target)
        s = {"X": X, "W": W, "target": target}
        if op == "ce_grad":
            s["lse"] = _logits_lse(X, W)
            s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
        return s
    M, N, K = case["M"], case["N"], case["K"]
    if op == "act_grad":
        return {"A": _normal(g, 1e-3, bf16, M, K), "B": _normal(g, K ** -0.5, bf16, K, N),
                "Z": _normal(g, 1.0, bf16, M, (2 if case["gated"] else 1) * N)}
    wide = (2 if case["gated"] else 1) * N
    s = {"A": _normal(g, 1.0, bf16, *((K, M) if case["trans_a"] else (M, K))),
         "B": _normal(g, K ** -0.5, bf16, *((wide, K) if case["trans_b"] else (K, wide))), "bias": None, "R": None}
    if case["bias"]:
        s["bias"] = _normal(g, 0.1, torch.float32, wide)
    if case["residual"]:
        s["R"] = _normal(g, 1.0, DTYPE[case["residual"]], M, N)
    return s


def prepare(case, seed):
    return dict(_inputs(case, seed), case=dict(case))


# ------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _apply(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z * _sigmoid(2.0 * ROOT_2_PI * (z + 0.044715 * z * z * z))
    return z * _sigmoid(z)


def _slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        s = _sigmoid(2.0 * ROOT_2_PI * (z + 0.044715 * z * z * z))
        return s + z * s * (1.0 - s) * (2.0 * ROOT_2_PI * (1.0 + 3.0 * 0.044715 * z * z))
    s = _sigmoid(z)
    return s + z * s * (1.0 - s)


def _left_out(target, V):
    return (target < 0) | (target >= V)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("ce", "ce_grad"):
        X, W, V = s["X"].float(), s["W"].float(), case["V"]
        out = _left_out(s["target"], V)
        at = torch.where(out, torch.zeros_like(s["target"]), s["target"])[:, None]
        z = X @ W.t()
        if op == "ce":
            m = z.amax(dim=1, keepdim=True)
            picked = z.gather(1, at)[:, 0]
            lse = m[:, 0] + torch.log(torch.exp(z - m).sum(dim=1))
            return {"loss": torch.where(out, torch.zeros_like(lse), lse - picked), "lse": lse}
        p = torch.exp(z - s["lse"][:, None])
        del z
        p.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
        p = torch.where(out[:, None], torch.zeros_like(p), p * s["dloss"][:, None])
        return {"dX": (p @ W).bfloat16(), "dW": (p.t() @ X).bfloat16()}
    if op == "act_grad":
        N = case["N"]
        d, z = s["A"].float() @ s["B"].float(), s["Z"].float()
        if case["gated"]:
            gate, up = z[:, :N], z[:, N:]
            dz = torch.cat((d * up * _slope(case["act"], gate), d * _apply(case["act"], gate)), dim=1)
        else:
            dz = d * _slope(case["act"], z)
        return {"dZ": dz.bfloat16(), "db": dz.sum(dim=0)}
    a = s["A"].float().t() if case["trans_a"] else s["A"].float()
    b = s["B"].float().t() if case["trans_b"] else s["B"].float()
    z = a @ b
    if s["bias"] is not None:
        z = z + s["bias"]
    N = case["N"]
    c = _apply(case["act"], z[:, :N]) * z[:, N:] if case["gated"] else _apply(case["act"], z)
    if s["R"] is not None:
        c = c + s["R"].float()
    out = {"C": c.to(DTYPE[case["type"]])}
    if case["keep_z"]:
        out["Z"] = z.bfloat16()
    return out


# ------------------------------------------------------- the framework's calls

def _framework(s):
    import tiled_matrix_multiplication_sm_gb300 as tg
    case = s["case"]
    op = case["op"]
    if op == "ce":
        loss, lse = tg.gemm_ce(s["X"], s["W"], s["target"])
        return {"loss": loss, "lse": lse}
    if op == "ce_grad":
        dx, dw = tg.gemm_ce_grad(s["X"], s["W"], s["target"], s["lse"], s["dloss"])
        return {"dX": dx, "dW": dw}
    if op == "act_grad":
        dz, db = tg.gemm_act_grad(s["A"], s["B"], s["Z"], case["act"], gated=case["gated"])
        return {"dZ": dz, "db": db}
    got = tg.gemm_act(s["A"], s["B"], case["act"], trans_a=case["trans_a"], trans_b=case["trans_b"], gated=case["gated"],
                      bias=s["bias"], residual=s["R"], keep_z=case["keep_z"], out_dtype=DTYPE[case["type"]])
    return {"C": got[0], "Z": got[1]} if case["keep_z"] else {"C": got}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------- work

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2, "": 0}
    if op in ("ce", "ce_grad"):
        T, V, D = case["T"], case["V"], case["D"]
        read = 2 * T * D + 2 * V * D + 8 * T
        if op == "ce":
            return {"bytes": read + 8 * T, "flops": 2 * T * V * D}
        return {"bytes": read + 8 * T + 2 * T * D + 2 * V * D, "flops": 6 * T * V * D}
    M, N, K = case["M"], case["N"], case["K"]
    wide = (2 if case["gated"] else 1) * N
    if op == "act_grad":
        return {"bytes": 2 * (M * K + K * N) + 4 * M * wide + 4 * wide, "flops": 2 * M * N * K}
    out = M * N * (size[case["type"]] + size[case["residual"]]) + (2 * M * wide if case["keep_z"] else 0)
    return {"bytes": 2 * (M * K + K * wide) + out + (4 * wide if case["bias"] else 0), "flops": 2 * M * wide * K}


# ------------------------------------------------------ 64-bit definitions

def _phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def _exact_act(act, z):
    """(act(z), act'(z))."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0.0), torch.where(z > 0, one, 0 * one)
    if act == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = ROOT_2_PI * (z + 0.044715 * z ** 3)
        h = (1 + torch.tanh(u)) / 2
        return z * h, h + z / 2 / torch.cosh(u.clamp(-300, 300)) ** 2 * ROOT_2_PI * (1 + 0.134145 * z ** 2)
    h = (1 + torch.tanh(z / 2)) / 2
    return z * h, h + z / 4 / torch.cosh((z / 2).clamp(-300, 300)) ** 2


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("ce", "ce_grad"):
        V = case["V"]
        X, W, target = s["X"].double(), s["W"].double(), s["target"]
        rows = torch.arange(len(target), device=target.device)
        kept = (target >= 0) & (target < V)
        z = torch.mm(X, W.T)
        if op == "ce":
            lse = torch.logsumexp(z, dim=1)
            loss = torch.zeros_like(lse)
            loss[kept] = lse[kept] - z[rows[kept], target[kept]]
            return {"loss": loss, "lse": lse}
        z.sub_(s["lse"].double()[:, None]).exp_()
        z[rows[kept], target[kept]] -= 1.0
        z.mul_(torch.where(kept, s["dloss"].double(), 0.0)[:, None])
        return {"dX": torch.mm(z, W), "dW": torch.mm(z.T, X)}
    if op == "act_grad":
        d, Z = torch.mm(s["A"].double(), s["B"].double()), s["Z"].double()
        if case["gated"]:
            gate, up = Z.chunk(2, dim=1)
            value, slope = _exact_act(case["act"], gate)
            dz = torch.hstack((d * slope * up, d * value))
        else:
            dz = d * _exact_act(case["act"], Z)[1]
        return {"dZ": dz, "db": torch.sum(dz, 0)}
    A, B = s["A"].double(), s["B"].double()
    z = torch.mm(A.T if case["trans_a"] else A, B.T if case["trans_b"] else B)
    if s["bias"] is not None:
        z += s["bias"].double()
    if case["gated"]:
        gate, up = z.chunk(2, dim=1)
        c = _exact_act(case["act"], gate)[0] * up
    else:
        c = _exact_act(case["act"], z)[0]
    out = {"C": c if s["R"] is None else c + s["R"].double()}
    if case["keep_z"]:
        out["Z"] = z
    return out
