"""One DeepSeekMoE layer forward, composed from the C-ABI calls.

The steps ("DeepSeek_V3_Report：Annotation", eqs. (12)-(16); quantise before
dispatch per "Low-Precision Communication"):

    moe_route -> moe_permute_index (counts, offsets, row maps, tile table)
      -> fp8_quant_1x128_scatter(u): each token quantised once, its FP8 row
         written in token order and at each of its K expert-sorted rows
      -> grouped GEMM 1 (W1, fused SwiGLU + 1x128 requantisation)
      -> grouped GEMM 2 (W2, fp32 rows) -> moe_combine -> moe_bias_update

All of it is queued on one CUDA stream with no host synchronisation: the
ragged expert segments travel through device-side offsets and the tile
table.  This module only owns buffers (torch allocations) and the call order;
every step runs in libmoefp8.so.

Row layout of the permuted activations (and of h and Y): rows [0, T*K) are
the routed pairs sorted by expert, rows [T*K, T*K+T) are the T tokens in
order, which the shared expert (group E of the grouped GEMMs) consumes.  The
quantiser writes the tokens into that tail and the routed rows in the same
pass, so neither the shared expert nor the dispatch costs a separate copy.
"""
from __future__ import annotations

import torch

from . import _abi
from .configs import MoEConfig
from . import inputs as _inputs


def reduce_load_counts(counts: torch.Tensor, tokens_per_rank: int, process_group=None):
    """Sum the per-expert routed-pair counts over the data-parallel ranks.

    The bias update needs the load of the whole batch ("Auxiliary-Loss-Free
    Load Balancing": loads are monitored over the whole batch of each step),
    so every rank applies the same +-gamma.  Returns (counts, total tokens)."""
    if process_group is None:
        return counts, tokens_per_rank
    import torch.distributed as dist
    total = counts.clone()
    dist.all_reduce(total, op=dist.ReduceOp.SUM, group=process_group)
    return total, tokens_per_rank * dist.get_world_size(process_group)


def reduce_weight_grads(grads: dict, process_group=None) -> dict:
    """Data parallelism: sum the fp32 expert weight gradients (dW1, dW2) and
    the centroids' (dcentroids) over the ranks in place, so every rank holds
    the gradient of the whole batch."""
    if process_group is None:
        return grads
    import torch.distributed as dist
    for k in ("dW1", "dW2", "dcentroids"):
        if k in grads:
            dist.all_reduce(grads[k], op=dist.ReduceOp.SUM, group=process_group)
    return grads


def max_over_ranks(value: float, device, process_group=None) -> float:
    """Largest value over the ranks (a time: the job finishes with its slowest rank)."""
    if process_group is None:
        return value
    import torch.distributed as dist
    t = torch.tensor([value], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX, group=process_group)
    return float(t.item())


def quantise_weight_stack(w_bf16: torch.Tensor, q=None, s=None, pow2: bool = False):
    """128x128 block quantisation of a [G][N][K] bf16 stack on the device."""
    return _abi.fp8_quant_128x128(w_bf16, q, s, pow2=pow2)


def make_fp8_weights(cfg: MoEConfig, device, chunk: int = 16, pow2: bool = False,
                     experts: list[int] | None = None):
    """Draw the bf16 expert weights (seeded, per expert) and quantise them on
    the device a few experts at a time; only the FP8 stacks stay resident.
    ``pow2`` rounds the block scales up to powers of two (for a layer built
    with pow2=True).  ``experts`` selects the stacked experts, in order
    (default: all routed experts, then the shared one = index E); an
    expert-parallel rank takes its own block plus the shared expert."""
    ids = list(range(cfg.E + cfg.n_shared)) if experts is None else list(experts)
    G = len(ids)
    w1q = torch.empty(G, 2 * cfg.I, cfg.d, dtype=torch.uint8, device=device)
    w1s = torch.empty(G, 2 * cfg.I // 128, cfg.d // 128, dtype=torch.float32, device=device)
    w2q = torch.empty(G, cfg.d, cfg.I, dtype=torch.uint8, device=device)
    w2s = torch.empty(G, cfg.d // 128, cfg.I // 128, dtype=torch.float32, device=device)
    for e0 in range(0, G, chunk):
        e1 = min(G, e0 + chunk)
        w1 = torch.stack([_inputs.draw_w1(cfg, ids[e], device) for e in range(e0, e1)])
        w2 = torch.stack([_inputs.draw_w2(cfg, ids[e], device) for e in range(e0, e1)])
        _abi.fp8_quant_128x128(w1, w1q[e0:e1], w1s[e0:e1], pow2=pow2)
        _abi.fp8_quant_128x128(w2, w2q[e0:e1], w2s[e0:e1], pow2=pow2)
        del w1, w2
    return w1q, w1s, w2q, w2s


class MoELayer:
    """Device buffers and call sequence of one layer for a fixed batch size T.

    ``pow2`` selects the power-of-two scale variant: the activations and h are
    quantised with scales rounded up to powers of two and both expert GEMMs
    hand the scales to the tensor core (grouped_gemm_fp8_pow2); the weights
    must come from make_fp8_weights(..., pow2=True).

    ``router_grad`` makes forward_train keep what the router's gradient needs
    (the logits, and the expert outputs as an 8-bit checkpoint) and backward
    include the router: du then holds its share too, and the centroids'
    gradient is returned.  backward then refuses to mix two passes: the last
    one has to be forward_train."""

    def __init__(self, cfg: MoEConfig, centroids: torch.Tensor, bias: torch.Tensor,
                 w1q, w1s, w2q, w2s, T: int | None = None, process_group=None,
                 keep_logits: bool = False, pow2: bool = False, balance_loss: bool = False,
                 seq_len: int | None = None, alpha: float = 1e-4, router_grad: bool = False):
        self.cfg = cfg
        self.router_grad = router_grad
        keep_logits = keep_logits or router_grad
        self.pow2 = pow2
        self.T = cfg.T if T is None else T
        self.dev = centroids.device
        self.centroids = centroids
        self.bias = bias
        self.w1q, self.w1s, self.w2q, self.w2s = w1q, w1s, w2q, w2s
        self.pg = process_group
        T, d, K, E, I = self.T, cfg.d, cfg.K, cfg.E, cfg.I
        P = T * K
        self.pairs = P
        dev = self.dev
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        self.idx = torch.empty(T, K, dtype=i32, device=dev)
        # router logits of the last step (keep_logits), and the sequence-wise
        # balance loss the router's selection pass computes (balance_loss:
        # sequences of seq_len tokens, default one sequence of T)
        self.logits = torch.empty(T, E, dtype=f32, device=dev) if keep_logits else None
        self.balance = (_abi.BalanceLossState(T, E, T if seq_len is None else seq_len, alpha,
                                              with_fp=True, device=dev)
                        if balance_loss else None)
        self.gate = torch.empty(T, K, dtype=f32, device=dev)
        self.route_ws = torch.empty(max(_abi.moe_route_workspace_size(T, d, E), 16), dtype=u8, device=dev)
        self.Xq = torch.empty(P + T, d, dtype=u8, device=dev)
        self.Xs = torch.empty(P + T, d // 128, dtype=f32, device=dev)
        self.perm = {
            "xq_perm": self.Xq[:P], "xs_perm": self.Xs[:P],
        }
        self.perm_ws = torch.empty(max(_abi.moe_permute_workspace_size(T, K, E), 16), dtype=u8, device=dev)
        self.H = torch.empty(P + T, I, dtype=u8, device=dev)
        self.Hs = torch.empty(P + T, I // 128, dtype=f32, device=dev)
        self.Y = torch.empty(P + T, d, dtype=f32, device=dev)
        self.out = torch.empty(T, d, dtype=f32, device=dev)
        self.dev_err = torch.zeros(1, dtype=i32, device=dev)
        # whether idx, gate, logits and the tables are the last forward_train's
        self._trained = False
        # the grouped GEMMs' work counter (dynamic tile scheduling)
        self.sched = torch.zeros(1, dtype=i32, device=dev)
        self.u_dev = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
        # second input/output pair and copy streams for forward_host_stream
        self._u_dev2 = None
        self._out2 = None
        self._streams = None
        # first permute allocates the index/tile buffers inside self.perm
        self.max_tiles = _abi.moe_max_m_tiles(T, K, E, True)

    # -- individual steps (also used by the benchmark to time them) --------
    def step_route(self, u):
        c = self.cfg
        self._trained = False                # what follows belongs to another pass
        _abi.moe_route(u, self.centroids, self.bias, c.G, c.M, c.K, self.idx, self.gate,
                       logits_out=self.logits, ws=self.route_ws, dev_err=self.dev_err,
                       aux=self.balance)

    def step_permute(self):
        """Counts, offsets, row maps and the tile table (no row moves yet)."""
        _abi.moe_permute_index(self.idx, self.cfg.E, True, out=self.perm, ws=self.perm_ws,
                               dev_err=self.dev_err)

    def step_quant(self, u):
        """1x128 quantisation of u, written in token order (the shared
        expert's rows) and at every routed row (the dispatch)."""
        P = self.pairs
        _abi.fp8_quant_1x128_scatter(u, self.perm["dst_of"], self.Xq[:P], self.Xs[:P],
                                     self.Xq[P:], self.Xs[P:], pow2=self.pow2)

    def step_gemm1(self):
        p = self.perm
        _abi.grouped_gemm_fp8_blockscaled(self.Xq, self.Xs, self.w1q, self.w1s, p["offsets"],
                                          p["tile_group"], p["tile_start"], p["n_tiles"],
                                          self.max_tiles, _abi.EP_SWIGLU_QUANT, self.H, self.Hs,
                                          dev_err=self.dev_err, pow2=self.pow2, sched=self.sched)

    def step_gemm2(self):
        p = self.perm
        _abi.grouped_gemm_fp8_blockscaled(self.H, self.Hs, self.w2q, self.w2s, p["offsets"],
                                          p["tile_group"], p["tile_start"], p["n_tiles"],
                                          self.max_tiles, _abi.EP_F32, self.Y,
                                          dev_err=self.dev_err, pow2=self.pow2, sched=self.sched)

    def step_combine(self, u, out=None):
        P = self.pairs
        _abi.moe_combine(self.Y, self.perm["dst_of"], self.gate, self.Y[P:], u,
                         self.out if out is None else out)

    def step_bias_update(self):
        counts, T_all = reduce_load_counts(self.perm["counts"], self.T, self.pg)
        _abi.moe_bias_update(counts, T_all, self.cfg.K, self.cfg.gamma, self.bias)

    # -- whole layer --------------------------------------------------------
    def forward(self, u: torch.Tensor, update_bias: bool = True,
                out: torch.Tensor | None = None) -> torch.Tensor:
        """u bf16 [T][d] on the device -> out fp32 [T][d] (self.out unless
        ``out`` is given)."""
        assert u.shape == (self.T, self.cfg.d) and u.dtype == torch.bfloat16
        out = self.out if out is None else out
        self.step_route(u)
        self.step_permute()
        self.step_quant(u)
        self.step_gemm1()
        self.step_gemm2()
        self.step_combine(u, out)
        if update_bias:
            self.step_bias_update()
        return out

    # -- training: forward with the SwiGLU input cached, and the backward ---
    def forward_train(self, u: torch.Tensor, update_bias: bool = True) -> torch.Tensor:
        """forward() that also caches what the backward needs: the SwiGLU
        input gu in FP8 (1x128 tiles; "Low-Precision Activation"), besides the
        FP8 expert inputs Xq and the routing that forward() keeps anyway.
        GEMM 1 writes gu in fp32, which is quantised for the cache and
        through SwiGLU for h.  With router_grad also the logits, the 8-bit
        checkpoint of the expert outputs, and u itself (not copied: it must
        keep its values until backward)."""
        assert u.shape == (self.T, self.cfg.d) and u.dtype == torch.bfloat16
        c = self.cfg
        rows = self.pairs + self.T
        if getattr(self, "GU", None) is None:
            dev = self.dev
            self.GU = torch.empty(rows, 2 * c.I, dtype=torch.float32, device=dev)
            self.GUq = torch.empty(rows, 2 * c.I, dtype=torch.uint8, device=dev)
            self.GUs = torch.empty(rows, 2 * c.I // 128, dtype=torch.float32, device=dev)
        self.step_route(u)
        self.step_permute()
        self.step_quant(u)
        p = self.perm
        _abi.grouped_gemm_fp8_blockscaled(self.Xq, self.Xs, self.w1q, self.w1s, p["offsets"],
                                          p["tile_group"], p["tile_start"], p["n_tiles"],
                                          self.max_tiles, _abi.EP_F32, self.GU,
                                          dev_err=self.dev_err, pow2=self.pow2)
        _abi.fp8_quant_1x128_f32(self.GU, self.pow2, self.GUq, self.GUs)
        _abi.swiglu_quant(self.GU, c.I, self.H, self.Hs, pow2=self.pow2)
        self.step_gemm2()
        if self.router_grad:
            self.step_combine_checkpoint(u)
            self._u_train = u
        else:
            self.step_combine(u, self.out)
        if update_bias:
            self.step_bias_update()
        self._trained = True
        return self.out

    def step_combine_checkpoint(self, u):
        """The combine that also leaves the routed expert outputs in 8 bits
        (Yq, Ys), which is all the backward needs of Y."""
        P = self.pairs
        if getattr(self, "Yq", None) is None:
            self.Yq = torch.empty(P, self.cfg.d, dtype=torch.uint8, device=self.dev)
            self.Ys = torch.empty(P, self.cfg.d // 128, dtype=torch.float32, device=self.dev)
        _abi.moe_combine_checkpoint(self.Y[:P], self.perm["dst_of"], self.gate, self.Y[P:], u,
                                    self.out, self.Yq, self.Ys, pow2=self.pow2,
                                    dev_err=self.dev_err)

    def transposed_weights(self):
        """The Dgrad GEMMs' B operands: W1^T [G][d][2I] and W2^T [G][I][d]
        with their block scales (made once per weight version)."""
        if getattr(self, "_wt", None) is None:
            w1t, w1ts = _abi.fp8_transpose_128x128(self.w1q, self.w1s)
            w2t, w2ts = _abi.fp8_transpose_128x128(self.w2q, self.w2s)
            self._wt = (w1t, w1ts, w2t, w2ts)
        return self._wt

    def backward(self, dout: torch.Tensor, weight_grads: bool = True, mark=None,
                 dbalance: torch.Tensor | None = None) -> dict:
        """Gradients of the expert FFNs for the upstream gradient dout (fp32
        [T][d]) of the last forward_train: du (the layer input's gradient
        through the residual and the experts; with router_grad through the
        router as well), and with weight_grads dW1 [G][2I][d], dW2 [G][d][I].
        With router_grad also dgate [T][K], dlogits [T][E] and (weight_grads)
        dcentroids [E][d]; dbalance (fp32, one value per sequence) is the
        upstream gradient of the balance loss of a layer built with
        balance_loss, None where the loss is not trained.
        A forward in between overwrites the routing: with router_grad that is
        refused.  Replays of captured calls are not seen here: capture
        forward_train and backward together.
        Dgrad: dy (1x128 FP8) . W2 -> dh; SwiGLU backward on the cached FP8
        gu -> dgu (1x128 FP8); dgu . W1 -> dx; un-permute.  Wgrad: the
        token-major 128x1 operands dy^T, h^T (recomputed), dgu^T, x^T through
        grouped_gemm_fp8_wgrad."""
        c = self.cfg
        p = self.perm
        mark = mark or (lambda name: None)
        if dbalance is not None and not (self.router_grad and self.balance is not None):
            raise _abi.MoEError("backward: dbalance needs a layer built with router_grad and balance_loss")
        if self.router_grad and not self._trained:
            raise _abi.MoEError("backward: the last pass of this layer was not forward_train: its routing, and "
                                "what the router's gradient needs, are gone")
        w1t, w1ts, w2t, w2ts = self.transposed_weights()
        dgate = None
        if self.router_grad:
            dyq, dys, dy, dgate = _abi.moe_combine_checkpoint_backward(
                dout, p["dst_of"], self.gate, self.Yq, self.Ys, want_dy=weight_grads,
                dev_err=self.dev_err)
        else:
            dyq, dys, dy = _abi.moe_combine_backward(dout, p["dst_of"], self.gate, want_dy=weight_grads)
        mark("combine_backward")
        dh = _abi.grouped_gemm_fp8_blockscaled(dyq, dys, w2t, w2ts, p["offsets"], p["tile_group"],
                                               p["tile_start"], p["n_tiles"], self.max_tiles,
                                               _abi.EP_F32, dev_err=self.dev_err, pow2=self.pow2)
        mark("dgrad2")
        dguq, dgus, dgu, h = _abi.swiglu_backward(dh, self.GUq, self.GUs, want_fp32=weight_grads)
        mark("swiglu_backward")
        dx = _abi.grouped_gemm_fp8_blockscaled(dguq, dgus, w1t, w1ts, p["offsets"], p["tile_group"],
                                               p["tile_start"], p["n_tiles"], self.max_tiles,
                                               _abi.EP_F32, dev_err=self.dev_err, pow2=self.pow2)
        mark("dgrad1")
        du = _abi.moe_unpermute_add(dx, p["dst_of"], dout)
        mark("unpermute")
        dlogits = dcentroids = None
        if self.router_grad:
            b = self.balance
            with_balance = dbalance is not None
            dlogits, du, dcentroids = _abi.moe_route_backward(
                dgate, self.logits, self.idx, self.gate, self._u_train, self.centroids, du_base=du,
                du=du, f=b.f[:b.n_seq] if with_balance else None, dloss=dbalance,
                alpha=b.alpha if with_balance else 0.0, seq_len=b.seq_len if with_balance else 0,
                want_dcentroids=weight_grads, dev_err=self.dev_err)
            mark("route_backward")
        r = {"du": du, "dyq": dyq, "dys": dys, "dh": dh, "dguq": dguq, "dgus": dgus, "dx": dx}
        if self.router_grad:
            r.update({"dgate": dgate, "dlogits": dlogits})
            if weight_grads:
                r["dcentroids"] = dcentroids
        if weight_grads:
            G = c.E + c.n_shared
            tabs = (p["offsets"], p["tile_group"], p["tile_start"], p["n_tiles"], self.max_tiles)
            dyt = _abi.fp8_quant_128x1_pow2(dy, *tabs)
            ht = _abi.fp8_quant_128x1_pow2(h, *tabs)
            dgut = _abi.fp8_quant_128x1_pow2(dgu, *tabs)
            xt = _abi.fp8_quant_128x1_pow2(self.Xq, *tabs, src_scale=self.Xs)
            mark("quant_128x1")
            r["dW2"] = _abi.grouped_gemm_fp8_wgrad(dyt[0], dyt[2], ht[0], ht[2], p["tile_start"], G,
                                                   dev_err=self.dev_err)
            mark("wgrad2")
            r["dW1"] = _abi.grouped_gemm_fp8_wgrad(dgut[0], dgut[2], xt[0], xt[2], p["tile_start"], G,
                                                   dev_err=self.dev_err)
            mark("wgrad1")
            r.update({"dy": dy, "dgu": dgu, "h": h, "dyt": dyt, "ht": ht, "dgut": dgut, "xt": xt})
            reduce_weight_grads(r, self.pg)
        return r

    def forward_host(self, u_host: torch.Tensor, out_host: torch.Tensor,
                     update_bias: bool = True) -> torch.Tensor:
        """End-to-end call with host buffers: copy u in (pinned host ->
        device), run the layer, copy the output back (device -> pinned host)."""
        self.u_dev.copy_(u_host, non_blocking=True)
        self.forward(self.u_dev, update_bias)
        out_host.copy_(self.out, non_blocking=True)
        return out_host

    def seq_balance_loss(self, seq_len: int | None = None, alpha: float | None = None,
                         with_fp: bool = False):
        """The complementary sequence-wise balance loss (eqs. 17-20) of the
        last step's routing, per sequence of seq_len tokens.  With
        balance_loss=True the router's selection pass has already computed it
        (for the seq_len and alpha the layer was built with); with
        keep_logits=True it is computed from the kept logits."""
        b = self.balance
        if b is not None:
            assert seq_len in (None, b.seq_len) and alpha in (None, b.alpha), \
                "the fused loss uses the layer's seq_len and alpha"
            loss = b.loss[:b.n_seq]
            return (loss, b.f[:b.n_seq], b.P[:b.n_seq]) if with_fp else loss
        assert self.logits is not None, "build the layer with balance_loss or keep_logits"
        return _abi.moe_seq_balance_loss(self.logits, self.cfg.K, self.T if seq_len is None
                                         else seq_len, 1e-4 if alpha is None else alpha, with_fp)

    def capture(self, u: torch.Tensor, update_bias: bool = True):
        """Record one forward step on the device input ``u`` (bf16 [T][d];
        the graph keeps its address, so refill it in place) into a CUDA
        graph.  ``graph.replay()`` then queues the whole layer -- every
        kernel, in order, on the current stream -- with one host call.  One
        eager step runs first (it sets the kernels' launch attributes and
        allocates the permutation's tables), so the bias is updated once.
        Single GPU: the multi-rank bias update holds a collective.
        Returns (graph, kernels per replay)."""
        assert self.pg is None, "capture() is single-GPU"
        side = torch.cuda.Stream(self.dev)
        side.wait_stream(torch.cuda.current_stream(self.dev))
        with torch.cuda.stream(side):
            self.forward(u, update_bias)
        torch.cuda.current_stream(self.dev).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        n0 = _abi.launch_count
        with torch.cuda.graph(graph):
            self.forward(u, update_bias)
        return graph, _abi.launch_count - n0

    def forward_host_stream(self, u_hosts, out_hosts, update_bias: bool = True):
        """End-to-end calls over a sequence of batches in pinned host memory
        (u_hosts[i] bf16 [T][d] -> out_hosts[i] fp32 [T][d]), with the copies
        overlapped: batch i+1's host->device copy and batch i-1's
        device->host copy run on their own streams while batch i computes on
        the current stream.  Two device input and output buffers alternate;
        each batch's layer steps (and its bias update) run in order on the
        current stream.  Returns out_hosts once every copy has been queued;
        the caller synchronises (or waits on the current stream, which is
        made to wait for the last copies)."""
        import torch as _t
        assert len(u_hosts) == len(out_hosts)
        if self._u_dev2 is None:
            self._u_dev2 = [self.u_dev, _t.empty_like(self.u_dev)]
            self._out2 = [self.out, _t.empty_like(self.out)]
            self._streams = (_t.cuda.Stream(self.dev), _t.cuda.Stream(self.dev))
        s_in, s_out = self._streams
        comp = _t.cuda.current_stream(self.dev)
        start = _t.cuda.Event()
        start.record(comp)
        in_ready = [None, None]    # input buffer b holds batch data
        comp_done = [start, start]  # compute that last read u_dev2[b] / wrote out2[b]
        out_read = [start, start]  # device->host copy that last read out2[b]
        for i, (uh, oh) in enumerate(zip(u_hosts, out_hosts)):
            b = i & 1
            with _t.cuda.stream(s_in):
                s_in.wait_event(comp_done[b])  # the batch before last is done with u_dev2[b]
                self._u_dev2[b].copy_(uh, non_blocking=True)
                in_ready[b] = _t.cuda.Event()
                in_ready[b].record(s_in)
            comp.wait_event(in_ready[b])
            comp.wait_event(out_read[b])      # out2[b] has been copied out
            self.forward(self._u_dev2[b], update_bias, out=self._out2[b])
            comp_done[b] = _t.cuda.Event()
            comp_done[b].record(comp)
            with _t.cuda.stream(s_out):
                s_out.wait_event(comp_done[b])
                oh.copy_(self._out2[b], non_blocking=True)
                out_read[b] = _t.cuda.Event()
                out_read[b].record(s_out)
        comp.wait_event(out_read[0])
        comp.wait_event(out_read[1])
        return out_hosts

    def check(self) -> None:
        """Raise if a kernel recorded a device-side error (synchronises)."""
        _abi.raise_dev_err(self.dev_err)
