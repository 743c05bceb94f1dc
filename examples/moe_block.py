"""A mixture-of-experts block on the library's operators, served and trained.

    python -m examples.moe_block

Serving: router -> experts' layer (with the block's residual) -> dense layer with bias, activation and residual,
for up to 64 tokens, captured in a CUDA graph. Prefill: norm -> router -> tokens sorted by expert -> grouped product ->
gated activation -> grouped product -> weighted sum, for any number of tokens, captured too. Training: the same block's
forward and backward pass, its activations kept in 8 bits; a dense layer's; and a router's, each fitted to a fixed task.
Plain PyTorch does the router's own projection, the losses and the updates.
"""
from __future__ import annotations

import argparse

import torch

import moe_grouped_gemm_tma_gb300 as dg
from moe_grouped_gemm_tma_gb300.inputs import quantize_128x128


def quantise(x, transpose=False):
    """bf16 [M,N] as e4m3 codes with 1x128 scales, along N or (transpose) along M of its transpose [N,M]."""
    M, N = x.shape
    rows, cols = (N, (M + 127) // 128 * 128) if transpose else (M, N)
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty(rows, cols // 128, dtype=torch.float32, device=x.device)
    if transpose:
        dg.dg_epilogue_backward(x, None, None, None, q, s, None)
    else:
        dg.dg_epilogue_backward(x, None, q, s, None, None, None)
    return q, s


class Block:
    """x + experts(x), then h + gelu(W h + b): decode for up to 64 tokens."""

    def __init__(self, H, I, E, k, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.I, self.E, self.k = H, I, E, k
        self.router = (torch.randn(E, H, generator=g, device=device) / H ** 0.5).bfloat16()
        self.W13, self.s13 = self._weights(g, E, 2 * I, H)
        self.W2, self.s2 = self._weights(g, E, H, I)
        W, s = self._weights(g, 1, H, H)
        self.W, self.s = W[0], s[0]
        self.bias = torch.randn(H, generator=g, device=device) * 0.1
        self.workspace = dg.moe_layer_workspace(64, k, E, H, I, device)

    @staticmethod
    def _weights(g, E, N, K):
        w = torch.randn(E * N, K, generator=g, device=g.device) / K ** 0.5
        q, s = quantize_128x128(w)          # (N is a multiple of 128: no scale block spans two experts)
        return q.view(E, N, K), s.view(E, N // 128, K // 128)

    def decode(self, x):
        """One step for the tokens x, bf16 [T,H]."""
        T = x.shape[0]
        ids = torch.empty(T, self.k, dtype=torch.int32, device=x.device)
        weights = torch.empty(T, self.k, dtype=torch.float32, device=x.device)
        dg.dg_moe_route(x @ self.router.t(), ids, weights)
        h = torch.empty_like(x)
        dg.dg_moe_layer(x, ids, weights, self.W13, self.s13, self.W2, self.s2, h, self.workspace, act="silu", residual=x)
        q, s = quantise(h)
        out = torch.empty_like(h)
        dg.dg_gemm_fp8_nt_epilogue(q, s, self.W, self.s, out, bias=self.bias, act="gelu", residual=h)
        return out

    def graph(self, T):
        """(x, out, graph): a captured step; write the tokens into x, replay the graph, read out."""
        x = torch.zeros(T, self.H, dtype=torch.bfloat16, device=self.bias.device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.decode(x)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        g.block = self                    # whose weights it reads: they live as long as it does
        with torch.cuda.graph(g):
            out = self.decode(x)
        return x, out, g


class Dense:
    """y = act(W x + b) + x with FP32 master weights, its products in FP8."""

    def __init__(self, H, act="gelu_tanh", seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.act, self.H = act, H
        self.master = torch.randn(H, H, generator=g, device=device) / H ** 0.5
        self.bias = torch.zeros(H, device=device)
        self.dW, self.dbias = torch.empty_like(self.master), torch.empty_like(self.bias)
        self.workspace = None

    def forward(self, x):
        self.W, self.s = quantize_128x128(self.master)
        q, s = quantise(x)
        self.xt = quantise(x, transpose=True)
        self.Z, y = torch.empty_like(x), torch.empty_like(x)
        return dg.dg_gemm_fp8_nt_epilogue(q, s, self.W, self.s, y, bias=self.bias, act=self.act, residual=x, Z=self.Z)

    def backward(self, dy):
        """dW and dbias from dy = dloss/dy; returns dloss/dx."""
        M, N = dy.shape
        Mp = (M + 127) // 128 * 128
        if self.workspace is None or self.workspace.numel() < dg.load().dg_epilogue_backward_workspace(M, N):
            self.workspace = dg.epilogue_backward_workspace(M, N, dy.device)
        q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=dy.device)
        qt = torch.empty(N, Mp, dtype=torch.float8_e4m3fn, device=dy.device)
        s = torch.empty(M, N // 128, device=dy.device)
        st = torch.empty(N, Mp // 128, device=dy.device)
        dg.dg_epilogue_backward(dy, self.Z, q, s, qt, st, self.dbias, self.workspace, act=self.act)
        dx = torch.empty_like(dy)
        # W is stored [out, in]: as the second operand of dZ . W it is MN-major, its scales transposed
        dg.dg_gemm_fp8(q, s, self.W, self.s.t().contiguous(), dx, b_mn_major=True)
        dg.dg_wgrad_fp8_nt(qt, st, *self.xt, self.dW, accumulate=False)
        return dx.add_(dy)

    def step(self, rate):
        self.master -= rate * self.dW
        self.bias -= rate * self.dbias


def train_dense(H=512, tokens=300, steps=60, rate=0.25, seed=0):
    """Fit a layer to another one of its kind; the losses."""
    teacher, layer = Dense(H, seed=seed + 1), Dense(H, seed=seed + 2)
    teacher.bias.normal_(generator=torch.Generator(device="cuda").manual_seed(seed + 3))
    x = torch.randn(tokens, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()
    target = teacher.forward(x).float()
    losses = []
    for _ in range(steps):
        diff = layer.forward(x).float() - target
        losses.append(float((diff * diff).mean()))
        # (the mean over tokens only, so that the gradient's size does not depend on the width)
        layer.backward((diff / tokens).bfloat16())
        layer.step(rate)
    return losses


class Experts:
    """x + experts(norm(x)) with FP32 master weights, for any number of tokens, its products in FP8. What is kept for the
    backward pass besides x: the experts' rows and their pre-activations in e4m3, the router's and the experts' outputs."""

    def __init__(self, H, I, E, k, act="silu", seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.I, self.E, self.k, self.act, self.eps = H, I, E, k, act, 1e-6
        self.norm = torch.ones(H, device=device)
        self.router = torch.randn(E, H, generator=g, device=device) / H ** 0.5
        self.master13 = torch.randn(E, 2 * I, H, generator=g, device=device) / H ** 0.5
        self.master2 = torch.randn(E, H, I, generator=g, device=device) / I ** 0.5
        self.weights = None
        self.update()

    def update(self):
        """The products' weights from the master weights, in the same memory each time, where captured passes read them. (A 128x128
        block's codes and scale are its transpose's too, which the backward pass multiplies by.)"""
        def codes(w):
            e, n, k = w.shape
            q, s = quantize_128x128(w.reshape(e * n, k))
            q, s = q.view(e, n, k), s.view(e, n // 128, k // 128)
            return [q, s, q.transpose(1, 2).contiguous(), s.transpose(1, 2).contiguous()]
        made = codes(self.master13) + codes(self.master2)
        if self.weights is None:
            self.weights = made
            self.W13, self.s13, self.W13t, self.s13t, self.W2, self.s2, self.W2t, self.s2t = made
        else:
            for old, new in zip(self.weights, made):
                old.copy_(new)

    def forward(self, x, rows_at_most=None):
        """The block's output for x, bf16 [T,H]. rows_at_most: rows of the grouped layout, known from the counts (None: as many as
        any routing needs, without a look at them)."""
        T, H, I, k, E, dev = x.shape[0], self.H, self.I, self.k, self.E, x.device
        e4m3, f32, bf16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
        new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        s = self.saved = {"x": x}
        s["y"], q, sf = new(T, H, dtype=bf16), new(T, H, dtype=e4m3), new(T, H // 128, dtype=f32)
        dg.dg_rmsnorm(x, self.norm, y=s["y"], q=q, sf=sf, eps=self.eps)
        s["logits"] = s["y"].float() @ self.router.t()
        s["ids"], s["weights"] = new(T, k, dtype=torch.int32), new(T, k, dtype=f32)
        dg.dg_moe_route(s["logits"], s["ids"], s["weights"])
        most = dg.moe_sort_rows(T, k, E)
        s["rows"], s["counts"], m_indices = new(T, k, dtype=torch.int32), new(E, dtype=torch.int32), new(most, dtype=torch.int32)
        dg.dg_moe_sort_contiguous(s["ids"], s["rows"], s["counts"], m_indices, dg.moe_sort_workspace(T, k, E, dev))
        M = most if rows_at_most is None else rows_at_most(s["counts"])
        s["m_indices"] = m_indices = m_indices[:M]
        s["A"], s["sfa"] = new(M, H, dtype=e4m3), new(M, H // 128, dtype=f32)
        dg.dg_moe_gather(q, sf, s["rows"], s["A"], s["sfa"], m_indices=m_indices)
        Z = new(M, 2 * I, dtype=bf16)
        dg.dg_m_grouped_contiguous(s["A"], s["sfa"], self.W13, self.s13, m_indices, Z)
        h, sh = new(M, I, dtype=e4m3), new(M, I // 128, dtype=f32)
        s["kept"], s["kept_sf"] = new(M, 2 * I, dtype=e4m3), new(M, 2 * I // 128, dtype=f32)
        dg.dg_glu(Z, h, sh, kept=s["kept"], kept_sf=s["kept_sf"], m_indices=m_indices, act=self.act)
        s["Y"] = new(M, H, dtype=bf16)
        dg.dg_m_grouped_contiguous(h, sh, self.W2, self.s2, m_indices, s["Y"])
        out = new(T, H, dtype=bf16)
        return dg.dg_moe_combine(s["Y"], s["rows"], out, weights=s["weights"], residual=x)

    def graph(self, T):
        """(x, out, graph): the captured forward pass of T tokens. Its replays read the block's weights as they are then."""
        x = torch.zeros(T, self.H, dtype=torch.bfloat16, device=self.norm.device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(x)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        g.block = self                    # whose weights it reads: they live as long as it does
        with torch.cuda.graph(g):
            out = self.forward(x)
        return x, out, g

    def train_forward(self, x):
        """The forward pass in as many rows as the routing has, whose counts the weight gradients need on the host."""
        def rows(counts):
            self.ks = [(c + 127) // 128 * 128 for c in counts.tolist()]
            return max(128, sum(self.ks))
        return self.forward(x, rows)

    def backward(self, dout):
        """The gradients of norm, router, master13 and master2 (as d...) from dout = dloss/dout; returns dloss/dx."""
        s, H, I, E, dev = self.saved, self.H, self.I, self.E, dout.device
        T, M = dout.shape[0], s["A"].shape[0]
        e4m3, f32, bf16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
        new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=dev)  # noqa: E731
        both = lambda n: (new(M, n, dtype=e4m3), new(M, n // 128, dtype=f32), new(n, M, dtype=e4m3), new(n, M // 128, dtype=f32))  # noqa: E731
        dY, dweights = new(M, H, dtype=bf16), new(T, self.k, dtype=f32)
        dg.dg_moe_combine_backward(dout, s["rows"], dY, weights=s["weights"], y=s["Y"], dweights=dweights, m_indices=s["m_indices"])
        q, sf, qt, sft = both(H)
        dg.dg_epilogue_backward(dY, None, q, sf, qt, sft, None)
        dH = new(M, I, dtype=bf16)
        dg.dg_m_grouped_contiguous(q, sf, self.W2t, self.s2t, s["m_indices"], dH)
        z, sz, zt, szt = both(2 * I)
        ht, sht = new(I, M, dtype=e4m3), new(I, M // 128, dtype=f32)
        dg.dg_glu_backward(dH, z, sz, zt, szt, ht, sht, kept=s["kept"], kept_sf=s["kept_sf"], act=self.act)
        At, sat = new(H, M, dtype=e4m3), new(H, M // 128, dtype=f32)
        dg.dg_transpose_fp8(s["A"], s["sfa"], At, sat)
        self.dmaster2, self.dmaster13 = torch.zeros_like(self.master2), torch.zeros_like(self.master13)
        if sum(self.ks):
            dg.dg_k_grouped_wgrad(qt, sft, ht, sht, self.ks, self.dmaster2)
            dg.dg_k_grouped_wgrad(zt, szt, At, sat, self.ks, self.dmaster13)
        dA, dy = new(M, H, dtype=bf16), new(T, H, dtype=bf16)
        dg.dg_m_grouped_contiguous(z, sz, self.W13t, self.s13t, s["m_indices"], dA)
        dg.dg_moe_combine(dA, s["rows"], dy)
        dlogits = torch.empty_like(s["logits"])
        dg.dg_moe_route_backward(s["logits"], s["ids"], dweights, dlogits)
        self.drouter = dlogits.t() @ s["y"].float()
        dy = (dy.float() + dlogits @ self.router).to(bf16)
        self.dnorm, dx = torch.empty_like(self.norm), new(T, H, dtype=bf16)
        self.steps = {"dY": dY, "dweights": dweights, "dH": dH, "z": (z, sz), "zt": (zt, szt), "ht": (ht, sht), "dA": dA, "dy": dy,
                      "q": (q, sf), "qt": (qt, sft), "At": (At, sat)}
        return dg.dg_rmsnorm_backward(dy, s["x"], self.norm, dx, self.dnorm, dg.rmsnorm_backward_workspace(T, H, dev), dsum=dout, eps=self.eps)

    def step(self, rate):
        for name in ("norm", "router", "master13", "master2"):
            getattr(self, name).sub_(getattr(self, "d" + name), alpha=rate)
        self.update()


def train_experts(H=512, I=256, E=8, k=2, tokens=600, steps=30, rate=0.2, seed=0):
    """Fit a block of experts to another one; the losses."""
    teacher, block = Experts(H, I, E, k, seed=seed + 1), Experts(H, I, E, k, seed=seed + 2)
    x = torch.randn(tokens, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()
    target = teacher.forward(x).float()
    losses = []
    for _ in range(steps):
        diff = block.train_forward(x).float() - target
        losses.append(float((diff * diff).mean()))
        block.backward((diff / tokens).bfloat16())
        block.step(rate)
    return losses


def train_router(H=256, E=32, k=4, tokens=512, steps=60, rate=20.0, seed=0):
    """Teach a router to give weight to the experts of highest value; the mean values it collects."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, H, device="cuda", generator=g)
    value = torch.tanh(x @ torch.randn(H, E, device="cuda", generator=g) / H ** 0.5)
    w = torch.randn(H, E, device="cuda", generator=g) / H ** 0.5
    ids = torch.empty(tokens, k, dtype=torch.int32, device="cuda")
    weights = torch.empty(tokens, k, device="cuda")
    dlogits = torch.empty(tokens, E, device="cuda")
    means = []
    for _ in range(steps):
        logits = x @ w
        dg.dg_moe_route(logits, ids, weights, scoring="softmax", renormalize=False)
        taken = value.gather(1, ids.long())
        means.append(float((weights * taken).sum(1).mean()))
        dg.dg_moe_route_backward(logits, ids, -taken / tokens, dlogits, scoring="softmax", renormalize=False)
        w -= rate * (x.t() @ dlogits)
    return means


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=1024)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--topk", type=int, default=4)
    a = p.parse_args()
    block = Block(a.hidden, a.inter, a.experts, a.topk)
    for T in (1, 8, 64):
        x, out, g = block.graph(T)
        x.normal_()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(3):
            g.replay()
        start.record()
        for _ in range(20):
            g.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"decode, {T} tokens: {start.elapsed_time(end) / 20 * 1e3:.1f} us a step")
    experts = Experts(a.hidden, a.inter, a.experts, a.topk)
    for T in (512, 4096):
        x, out, g = experts.graph(T)
        x.normal_()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(3):
            g.replay()
        start.record()
        for _ in range(20):
            g.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"prefill, {T} tokens: {start.elapsed_time(end) / 20 * 1e3:.1f} us a step")
    losses = train_experts()
    print(f"experts: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    losses = train_dense()
    print(f"dense layer: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    means = train_router()
    print(f"router: mean value {means[0]:.4f} -> {means[-1]:.4f} in {len(means)} steps")
    if dg.dg_device_status():
        raise SystemExit("a kernel reported an error")


if __name__ == "__main__":
    main()
