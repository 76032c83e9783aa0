"""A trunk block in front of the cell, made of the trunk operators: pre-norm, a gated selective-scan
mixer with its short convolution, dropout into the residual stream, the next norm, and the CfC
K-loop on it.

    n  = norm(s)                                  [K, B, D]
    x, z = n W_in^T                               [K, B, E] each
    u  = conv(x);  dt, B, C = u W_p^T             [K, B, E], [K, B, G, N] twice
    y  = scan(u, dt, A, B, C, D, dt_bias, z)      [K, B, E]
    s' = s + dropout(y W_out^T);  n' = norm(s')
    H  = cell(n')                                 [K, B, C]

``TrunkBlock`` trains it (``forward`` / ``backward`` write every gradient), ``TrunkServe`` runs
prompts and then single tokens with carried states (no dropout, up to n').  The plain products are
torch's; everything else is this library's kernels.  All float32, as the cell.
"""
from __future__ import annotations

import torch

from . import _lib
from .step import KLoopStep
from .trunk import ConvStep, ConvToken, DropoutNormStep, LayerNormStep, ScanStep, ScanToken


def make_params(D: int, E: int, N: int, C: int, W: int = 4, G: int = 1, seed: int = 0,
                device=None) -> dict:
    """Random parameters of a block: D stream channels, E mixer channels, N states, W taps, C
    cell channels."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g) * std + mean

    p = dict(w1=normal(D, std=0.1, mean=1.0), b1=normal(D, std=0.1),
             W_in=normal(2 * E, D, std=D ** -0.5), conv_w=normal(E, W, std=W ** -0.5),
             conv_b=normal(E, std=0.1), W_p=normal(E + 2 * G * N, E, std=E ** -0.5),
             A=-torch.arange(1.0, N + 1).repeat(E, 1), D=normal(E, std=0.1, mean=1.0),
             dt_bias=normal(E, std=0.5, mean=-3.0), W_out=normal(D, E, std=E ** -0.5),
             w2=normal(D, std=0.1, mean=1.0), b2=normal(D, std=0.1),
             cell_W=normal(4, C, D + C, std=(D + C) ** -0.5), cell_b=normal(4, C, std=0.1))
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return {k: v.to(dev).contiguous() for k, v in p.items()}


class TrunkBlock:
    """One training step of the block for K steps of B sequences.  Like the steps it is made of, it
    owns its results: what forward and backward return is valid until they are called again (clone
    what has to outlive that, such as gradients that are summed over several steps)."""

    def __init__(self, K: int, B: int, params: dict, p_drop: float = 0.1, G: int = 1):
        self.K, self.B, self.G, self.params = K, B, G, params
        self.D, self.E = params["W_out"].shape
        self.N, self.W = params["A"].shape[1], params["conv_w"].shape[1]
        self.C = params["cell_b"].shape[1]
        rows = K * B
        self.norm = LayerNormStep(rows, self.D)
        self.conv = ConvStep(K, B, self.E, self.W)
        self.scan = ScanStep(K, B, self.E, self.N, G, train=True)
        self.drop = DropoutNormStep(rows, self.D, p_drop)
        self.cell = KLoopStep(B, K, self.C, self.D)
        # The backward pass of each step is bound when its gradient's buffer exists; these do.
        dev = self.norm.device
        self.dy = torch.empty(K, B, self.E, device=dev)
        self.du = torch.empty(K, B, self.E, device=dev)
        self.dn = torch.empty(rows, self.D, device=dev)

    def forward(self, s, h0, ts, rng, lengths=None) -> torch.Tensor:
        """H [K, B, C] from the stream s [K, B, D], the cell's h0 [B, C] and time scales ts
        [K, B]; rng is the dropout's device-side {seed, offset}."""
        P, K, B, E, GN = self.params, self.K, self.B, self.E, self.G * self.N
        self.s = s.reshape(K * B, self.D)
        self.norm.bind(self.s, P["w1"], P["b1"], self.dn).forward()
        self.xz = (self.norm.y @ P["W_in"].T).view(K, B, 2 * E)
        self.conv.bind(self.xz[..., :E], P["conv_w"], P["conv_b"], lengths=lengths,
                       dy=self.du).forward()
        self.p = self.conv.u @ P["W_p"].T
        bc = self.p[..., E:].unflatten(-1, (2, self.G, self.N))
        self.scan.bind(self.conv.u, self.p[..., :E], P["A"], bc[..., 0, :, :], bc[..., 1, :, :],
                       P["D"], P["dt_bias"], self.xz[..., E:], lengths=lengths,
                       dy=self.dy).forward()
        self.o = self.scan.y.view(K * B, E) @ P["W_out"].T
        self.h0, self.ts, self.rng = h0, ts, rng
        self.drop.bind(self.o, self.s, rng, P["w2"], P["b2"]).forward()
        self.u_cell = self.drop.y.view(K, B, self.D)
        _lib.cfc_forward(self.u_cell, h0, P["cell_W"], P["cell_b"], ts, self.cell.H,
                         self.cell.cache, ws=self.cell.fws)
        return self.cell.H

    def backward(self, dH) -> dict:
        """Gradients of sum dH . H: of every parameter (by its name), of the stream (ds) and of
        the cell's initial state (dh0)."""
        P, K, B, E, GN = self.params, self.K, self.B, self.E, self.G * self.N
        c = self.cell
        c.bind(self.u_cell, self.h0, P["cell_W"], P["cell_b"], self.ts, dH).backward()
        self.drop.bind(self.o, self.s, self.rng, P["w2"], P["b2"],
                       dy=c.du.view(K * B, self.D)).backward()
        do = self.drop.dx
        torch.mm(do, P["W_out"], out=self.dy.view(K * B, E))
        self.scan.backward()
        dbc = torch.stack([self.scan.dB, self.scan.dC], 2).view(K, B, 2 * GN)
        dp = torch.cat([self.scan.ddt, dbc], -1).view(K * B, E + 2 * GN)
        u = self.conv.u.view(K * B, E)
        torch.addmm(self.scan.dx.view(K * B, E), dp, P["W_p"], out=self.du.view(K * B, E))
        self.conv.backward()
        dxz = torch.cat([self.conv.dx, self.scan.dz], -1).view(K * B, 2 * E)
        torch.mm(dxz, P["W_in"], out=self.dn)
        self.norm.backward()
        return dict(w1=self.norm.dw, b1=self.norm.db, W_in=dxz.T @ self.norm.y,
                    conv_w=self.conv.dw, conv_b=self.conv.dbias, W_p=dp.T @ u, A=self.scan.dA,
                    D=self.scan.dD, dt_bias=self.scan.ddt_bias,
                    W_out=do.T @ self.scan.y.view(K * B, E), w2=self.drop.dw, b2=self.drop.db,
                    cell_W=c.dW, cell_b=c.db, dh0=c.dh0,
                    ds=(self.norm.dx + self.drop.dres).view(K, B, self.D))


class TrunkServe:
    """The block up to n' for serving: a prompt of any length, then single tokens, with the
    convolution's and the scan's states carried in place."""

    def __init__(self, B: int, params: dict, G: int = 1):
        self.B, self.G, self.params = B, G, params
        self.D, self.E = params["W_out"].shape
        self.N, self.W = params["A"].shape[1], params["conv_w"].shape[1]
        dev = params["A"].device
        self.conv_state = torch.zeros(B, self.W - 1, self.E, device=dev)
        self.state = torch.zeros(B, self.E, self.N, device=dev)
        self.norms = [LayerNormStep(B, self.D), LayerNormStep(B, self.D)]
        self.conv, self.scan = ConvToken(B, self.E, self.W), ScanToken(B, self.E, self.N, G)

    def prompt(self, s, lengths=None) -> torch.Tensor:
        """n' [K, B, D] of a prompt s [K, B, D], continuing from the carried states."""
        P, E = self.params, self.E
        K, B, D = s.shape
        rows = s.reshape(K * B, D)
        first = LayerNormStep(K * B, D).bind(rows, P["w1"], P["b1"])
        first.run()
        xz = (first.y @ P["W_in"].T).view(K, B, 2 * E)
        conv = ConvStep(K, B, E, self.W).bind(xz[..., :E], P["conv_w"], P["conv_b"],
                                              self.conv_state, lengths)
        conv.run()
        p = conv.u @ P["W_p"].T
        bc = p[..., E:].unflatten(-1, (2, self.G, self.N))
        scan = ScanStep(K, B, E, self.N, self.G).bind(
            conv.u, p[..., :E], P["A"], bc[..., 0, :, :], bc[..., 1, :, :], P["D"], P["dt_bias"],
            xz[..., E:], self.state, lengths)
        scan.run()
        self.conv_state.copy_(conv.last)
        self.state.copy_(scan.h)
        second = LayerNormStep(K * B, D).bind(rows + scan.y.view(K * B, E) @ P["W_out"].T, P["w2"],
                                              P["b2"])
        second.run()
        return second.y.view(K, B, D)

    def token(self, s) -> torch.Tensor:
        """n' [B, D] of one token s [B, D] per sequence, a tensor of its own as the prompt's is."""
        P, E = self.params, self.E
        self.norms[0].bind(s, P["w1"], P["b1"]).run()
        xz = self.norms[0].y @ P["W_in"].T
        u, _ = self.conv.bind(xz[:, :E], P["conv_w"], self.conv_state, P["conv_b"]).run()
        p = u @ P["W_p"].T
        bc = p[:, E:].unflatten(-1, (2, self.G, self.N))
        y, _ = self.scan.bind(u, p[:, :E], P["A"], bc[:, 0], bc[:, 1], self.state, P["D"],
                              P["dt_bias"], xz[:, E:]).run()
        last = self.norms[1]
        last.y = torch.empty_like(last.y)  # not the one that the caller has from the token before
        last.bind(s + y @ P["W_out"].T, P["w2"], P["b2"]).run()
        return last.y
