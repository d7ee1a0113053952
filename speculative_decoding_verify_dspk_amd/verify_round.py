"""One verify round on the GPU, composed from the C-ABI calls.

A round ("mlx-dspark" wiki summary, "Architecture"): every projection of the
target over the M rows (anchor + drafts, or B requests x rows), the vocabulary
head with the row argmax (or logits for sampling), and the acceptance step,
whose few result words the caller may have written straight into pinned host
memory ("mlx-dspark releases", v0.2.0 notes: at most one device sync per
round).

Weights and activations are seeded synthetic tensors of the workload's shapes
(``inputs.LAYER_SHAPES``).  Each decoder layer contributes four launches, as a
real layer's dependencies allow: q/k/v grouped (they read the same rows), o,
gate/up grouped, down.  The four inputs of a layer are independent N(0, 1)
rows; the residual stream's norms and the activation function are outside this
path.  With ``attach_cache`` a layer's attention is part of it: q and k are
normed per head and rotated, k and v stored in a paged cache, the rows attend
over it, and o reads what comes out; ``set_tree`` makes the rows a drafted tree
instead of a chain, and ``launch_commit`` moves the accepted path's entries
together after the acceptance.

``Int8VerifyStack`` is the same round over 8-bit integer layers, rows and weights
alike, with the parts between the projections: the residual stream and its norms, the
activation or a router and its experts.  There a layer reads what the layer before it
wrote.

A round's launches can be captured once into HIP graphs (``capture_round``)
and replayed every round: the kernels take no host-side work between calls
(their workspaces come back zeroed), so a replay is the whole round in one
submission, without host launch gaps between its kernels.
"""
from __future__ import annotations

from dataclasses import dataclass, field

from . import binding, inputs


@dataclass
class Layer:
    qkv: list
    o: binding.DeviceQWeight
    gateup: list
    down: binding.DeviceQWeight


HEAD_DIM = 128              # of every workload's layer


@dataclass
class VerifyStack:
    model: str
    n_layers: int
    bits: int
    max_m: int
    copies: int = 1
    seed: str = "stack"
    layers: list = field(default_factory=list)   # [copy][layer] -> Layer
    heads: list = field(default_factory=list)    # [copy] -> DeviceQWeight

    def __post_init__(self):
        import torch
        s = inputs.LAYER_SHAPES[self.model]
        self.hidden, self.qdim, self.kvdim, self.inter, self.vocab = (s["hidden"], s["q"], s["kv"], s["inter"],
                                                                      s["vocab"])
        H, Q, KV, F, V = self.hidden, self.qdim, self.kvdim, self.inter, self.vocab

        def mk(n, k, *lab):
            c, sc, bi = inputs.make_qweight_device(n, k, self.bits, self.model, self.seed, *lab)
            return binding.DeviceQWeight(n, k, self.bits, c, sc, bi)

        for cp in range(self.copies):
            ls = []
            for li in range(self.n_layers):
                ls.append(Layer(qkv=[mk(Q, H, cp, li, "q"), mk(KV, H, cp, li, "k"), mk(KV, H, cp, li, "v")],
                                o=mk(H, Q, cp, li, "o"),
                                gateup=[mk(F, H, cp, li, "gate"), mk(F, H, cp, li, "up")],
                                down=mk(H, F, cp, li, "down")))
            self.layers.append(ls)
            self.heads.append(mk(V, H, cp, "lm_head"))
        M = self.max_m
        act = lambda k, name: inputs.make_activations_device(M, k, self.model, self.seed, name)
        self.x_attn, self.x_o, self.x_mlp, self.x_down = act(H, "attn_in"), act(Q, "o_in"), act(H, "mlp_in"), \
            act(F, "down_in")
        self.h = act(H, "final_h")
        f32 = dict(dtype=torch.float32, device="cuda")
        self.y_qkv = [torch.empty((M, Q), **f32), torch.empty((M, KV), **f32), torch.empty((M, KV), **f32)]
        self.y_o = torch.empty((M, H), **f32)
        self.y_gu = [torch.empty((M, F), **f32), torch.empty((M, F), **f32)]
        self.y_down = torch.empty((M, H), **f32)
        self.argmax = torch.empty((M,), dtype=torch.int32, device="cuda")
        self.logits = torch.empty((M, V), **f32)
        # one workspace per launch shape (their split-K layouts differ)
        wsb = binding.qgemm_workspace_bytes
        self.ws_qkv = binding.alloc_workspace(wsb(Q, H, M) + 2 * wsb(KV, H, M))
        self.ws_o = binding.alloc_workspace(wsb(H, Q, M))
        self.ws_gu = binding.alloc_workspace(2 * wsb(F, H, M))
        self.ws_down = binding.alloc_workspace(wsb(H, F, M))
        self.ws_head = binding.alloc_workspace(binding.lmhead_workspace_bytes(V, M))

        self.caches = None
        self.tree_mask = self.positions = None

    # -------------------------------------------------------------- attention
    def attach_cache(self, context: int, bits: int = 16, page_tokens: int = 64, room: int = 0,
                     eps: float = 1e-6) -> None:
        """Gives every layer a k/v cache of one request holding ``context``
        synthetic entries, with room for max_m rows and ``room`` more positions
        after them; from then on the layers attend over it, the rows a chain."""
        import torch
        self.tree_mask = self.positions = None
        D = HEAD_DIM
        self.q_heads, self.kv_heads, self.eps = self.qdim // D, self.kvdim // D, eps
        pages = -(-(context + self.max_m + room) // page_tokens)
        g = inputs.device_generator(self.model, self.seed, "cache", context)
        self.page_table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        self.cache_len = torch.full((1,), context, dtype=torch.int32, device="cuda")
        f32 = lambda *z: torch.empty(z, dtype=torch.float32, device="cuda")
        self.caches, self.q_norm, self.k_norm = [], [], []
        if context:
            past = binding.AttnBatch(torch.zeros_like(self.cache_len), self.page_table, context)
        for _ in range(self.n_layers):
            c = binding.KVCache.alloc(pages, self.kv_heads, D, page_tokens, bits)
            if context:
                k, v = (f32(context, self.kvdim).normal_(generator=g) for _ in range(2))
                binding.kv_append(c, past, k, v)
            self.caches.append(c)
            self.q_norm.append(f32(D).uniform_(0.8, 1.2, generator=g))
            self.k_norm.append(f32(D).uniform_(0.8, 1.2, generator=g))
        self.inv_freq = (1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.q_rot = torch.empty((self.max_m, self.qdim), **bf)
        self.attn_out = torch.empty((self.max_m, self.qdim), **bf)
        self.mask_buf = torch.empty((1, self.max_m), dtype=torch.int64, device="cuda")
        i32 = lambda n: torch.zeros((1, n), dtype=torch.int32, device="cuda")
        self.position_buf, self.parent_buf, self.path = i32(self.max_m), i32(self.max_m), i32(self.max_m)
        self.ws_attn = binding.alloc_workspace(
            binding.attn_workspace_bytes(self.q_heads, self.kv_heads, D, 1, self.max_m))

    def set_tree(self, parents, m: int, stream=None) -> None:
        """The next rounds' rows are the nodes of a tree (parents: int32 [m - 1]
        on the device, see dspk_tree_layout); None: a chain again.  The parents
        are copied, into the same memory each time, so that captured rounds of m
        rows follow."""
        import torch
        if parents is None:
            self.tree_mask = self.positions = None
            return
        if not self.caches:
            raise ValueError("set_tree: a tree's rows attend over a cache (attach_cache)")
        if m < 1 or m > self.max_m:
            raise ValueError(f"set_tree: a tree of {m} nodes in a stack of {self.max_m} rows")
        binding._int32(parents, "parents", m - 1)
        with torch.cuda.stream(stream):
            self.parent_buf[:, :m - 1].copy_(parents.reshape(1, -1)[:, :m - 1])
        self.tree_mask, self.positions = self.mask_buf[:, :m], self.position_buf[:, :m]
        self._lay_out(stream)

    def _lay_out(self, stream=None) -> None:
        """Masks and positions of the tree at the cached length."""
        m = self.positions.shape[1]
        binding.tree_layout(self.parent_buf, 1, m, self.cache_len, self.tree_mask, self.positions, stream)

    def attention_calls(self, li: int, m: int, stream=None) -> list:
        """Layer li's calls between q/k/v and o, their arguments marshalled."""
        batch = binding.AttnBatch(self.cache_len, self.page_table, m)
        c = self.caches[li]
        pos = None if self.positions is None else self.positions.view(-1)
        mask = None if self.tree_mask is None else self.tree_mask.view(-1)
        return [binding.prepare_qkv_norm_rope_append(c, batch, *self.y_qkv, self.q_heads, self.q_rot,
                                                     q_weight=self.q_norm[li], k_weight=self.k_norm[li], eps=self.eps,
                                                     inv_freq=self.inv_freq, positions=pos, stream=stream),
                binding.prepare_tree_attention(c, batch, self.q_rot, self.q_heads, self.attn_out, self.ws_attn,
                                               tree_mask=mask, stream=stream)]

    def launch_commit(self, path, accept_len, m: int, stream=None) -> None:
        """After the acceptance of a tree of m nodes: the path's entries of every
        layer move together, the cached length grows by the accepted nodes, and
        the tree's positions follow it.
        (A chain's entries are in place: its cached length grows by accept_len.)"""
        binding.kv_commit(self.caches, binding.AttnBatch(self.cache_len, self.page_table, m), path, accept_len,
                          self.cache_len, stream)
        if self.tree_mask is not None:
            self._lay_out(stream)

    # ------------------------------------------------------------------ sizes
    def layer_weight_bytes(self) -> int:
        L = self.layers[0][0]
        return sum(w.nbytes for w in L.qkv + [L.o] + L.gateup + [L.down])

    def head_weight_bytes(self) -> int:
        return self.heads[0].nbytes

    def round_weight_bytes(self) -> int:
        return self.n_layers * self.layer_weight_bytes() + self.head_weight_bytes()

    # ---------------------------------------------------------------- launches
    def launch_layers(self, m: int, copy: int = 0, stream=None) -> None:
        for li, L in enumerate(self.layers[copy]):
            binding.qgemm_verify_grouped(L.qkv, self.x_attn, m, self.y_qkv, self.ws_qkv, stream)
            if self.caches:
                for call in self.attention_calls(li, m, stream):
                    call()
            binding.qgemm_verify(L.o, self.attn_out if self.caches else self.x_o, m, self.y_o, self.ws_o, stream)
            binding.qgemm_verify_grouped(L.gateup, self.x_mlp, m, self.y_gu, self.ws_gu, stream)
            binding.qgemm_verify(L.down, self.x_down, m, self.y_down, self.ws_down, stream)

    def launch_head(self, m: int, copy: int = 0, want_logits: bool = False, stream=None) -> None:
        binding.lmhead_argmax(self.heads[copy], self.h, m, self.argmax, self.logits if want_logits else None,
                              self.ws_head, stream)

    def prepare_round(self, m: int, copy: int, want_logits: bool = False, stream=None):
        """The round's projection and head calls at width m on weight copy
        ``copy`` with their arguments marshalled once: (layer calls, head call)."""
        layers = []
        for li, L in enumerate(self.layers[copy]):
            layers += [binding.prepare_qgemm_grouped(L.qkv, self.x_attn, m, self.y_qkv, self.ws_qkv, stream)]
            layers += self.attention_calls(li, m, stream) if self.caches else []
            layers += [binding.prepare_qgemm(L.o, self.attn_out if self.caches else self.x_o, m, self.y_o, self.ws_o,
                                             stream),
                       binding.prepare_qgemm_grouped(L.gateup, self.x_mlp, m, self.y_gu, self.ws_gu, stream),
                       binding.prepare_qgemm(L.down, self.x_down, m, self.y_down, self.ws_down, stream)]
        head = binding.prepare_lmhead(self.heads[copy], self.h, m, self.argmax, self.logits if want_logits else None,
                                      self.ws_head, stream)
        return layers, head

    def capture_calls(self, m: int, copy: int, accept, want_logits: bool = False):
        """HIP graphs (layers, head, accept) of one round at width m on weight
        copy ``copy``; ``accept`` launches the acceptance step.  Replay them in
        that order on one stream."""
        import torch
        fns = (lambda: self.launch_layers(m, copy),
               lambda: self.launch_head(m, copy, want_logits=want_logits),
               accept)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):          # one eager pass before capture
            for f in fns:
                f()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graphs = []
        for f in fns:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                f()
            graphs.append(g)
        return graphs

    def launch_accept(self, m: int, draft_ids, accept_len, committed, stream=None) -> None:
        """Greedy acceptance of one request of m rows: along the tree that is set
        (the accepted nodes go to ``path``), or of a chain."""
        if self.tree_mask is None:
            binding.accept_greedy(self.argmax, draft_ids, 1, m, accept_len, committed, stream)
        else:
            binding.accept_tree_greedy(self.argmax, draft_ids, self.parent_buf, 1, m, accept_len, committed, self.path,
                                       stream)

    def capture_round(self, m: int, copy: int, draft_ids, accept_len, committed):
        """HIP graphs (layers, head, accept) of one greedy round at width m, of a
        tree if one is set at the time."""
        return self.capture_calls(m, copy, lambda: self.launch_accept(m, draft_ids, accept_len, committed))


@dataclass
class Int8Layer:
    qkv: binding.Int8Weight                      # q, k and v by columns
    o: binding.Int8Weight
    gate_up: binding.Int8Weight | None = None    # gate and up by columns: a dense layer
    down: binding.Int8Weight | None = None
    moe: binding.MoEWeights | None = None        # or a router and its experts
    router: object = None
    attn_norm: object = None                     # float32 [hidden]
    mlp_norm: object = None


@dataclass
class Int8VerifyStack(VerifyStack):
    """A stack of 8-bit integer layers with the model's head (``bits`` is the head's
    format).  ``experts`` > 0: mixture layers, ``top_k`` of the experts for each row,
    each of width ``expert_inter``.

    A layer: residual += the rows before it, norm to 8 bits, q/k/v, the attention side
    (with attach_cache; else o reads rows of its own), its rows to 8 bits, o, residual
    and norm again, then gate and up, activation to 8 bits, down, or router and experts.
    After the last layer residual and norm give the head its bf16 rows."""
    experts: int = 0
    top_k: int = 0
    expert_inter: int = 0
    norm_eps: float = 1e-6

    def __post_init__(self):
        import torch
        s = inputs.LAYER_SHAPES[self.model]
        self.hidden, self.qdim, self.kvdim, self.inter, self.vocab = (s["hidden"], s["q"], s["kv"], s["inter"],
                                                                      s["vocab"])
        H, Q, KV, F, V, M = self.hidden, self.qdim, self.kvdim, self.inter, self.vocab, self.max_m
        if self.experts:
            F = self.expert_inter
            if not 1 <= self.top_k <= self.experts or F < 1:
                raise ValueError("experts: top_k of 1 .. experts and expert_inter >= 1 are needed")
        lab = (self.model, self.seed, "int8")
        mk = lambda *z: binding.Int8Weight(*inputs.make_int8_device(z[0], *lab, *z[1:]))
        f32 = dict(dtype=torch.float32, device="cuda")
        for cp in range(self.copies):
            ls = []
            for li in range(self.n_layers):
                g = inputs.device_generator(*lab, cp, li, "norm")
                norm = lambda: torch.empty(H, **f32).uniform_(0.8, 1.2, generator=g)
                L = Int8Layer(qkv=mk((Q + 2 * KV, H), cp, li, "qkv"), o=mk((H, Q), cp, li, "o"), attn_norm=norm(),
                              mlp_norm=norm())
                if self.experts:
                    L.moe = binding.MoEWeights(*(mk((self.experts,) + z, cp, li, name) for name, z in
                                                 (("gate", (F, H)), ("up", (F, H)), ("down", (H, F)))))
                    L.router = torch.empty((self.experts, H), **f32).normal_(0.0, H ** -0.5, generator=g).bfloat16()
                else:
                    L.gate_up, L.down = mk((2 * F, H), cp, li, "gate_up"), mk((H, F), cp, li, "down")
                ls.append(L)
            self.layers.append(ls)
            c, sc, bi = inputs.make_qweight_device(V, H, self.bits, *lab, cp, "lm_head")
            self.heads.append(binding.DeviceQWeight(V, H, self.bits, c, sc, bi))
        g = inputs.device_generator(*lab, "final_norm")
        self.final_norm = torch.empty(H, **f32).uniform_(0.8, 1.2, generator=g)
        act = lambda k, name: inputs.make_activations_device(M, k, self.model, self.seed, name).view(torch.bfloat16)
        self.x_in, self.x_o = act(H, "embedded"), act(Q, "o_in")
        bf, i8 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int8, device="cuda")
        codes = lambda k: (torch.zeros((M, -(-k // 16) * 16), **i8)[:, :k], torch.zeros(M, **f32))
        self.residual, self.h, self.normed = (torch.zeros((M, H), **bf) for _ in range(3))
        self.x8, self.o8, self.h8 = codes(H), codes(Q), codes(F)
        qkv = torch.zeros((M, Q + 2 * KV), **f32)
        self.qkv, self.y_qkv = qkv, [qkv[:, :Q], qkv[:, Q:Q + KV], qkv[:, Q + KV:]]
        self.y_o, self.y_down = torch.zeros((M, H), **f32), torch.zeros((M, H), **f32)
        self.gate_up = None if self.experts else torch.zeros((M, 2 * F), **bf)
        self.argmax = torch.empty((M,), dtype=torch.int32, device="cuda")
        self.logits = torch.empty((M, V), **f32)
        if self.experts:
            self.ids = torch.zeros((M, self.top_k), dtype=torch.int32, device="cuda")
            self.expert_weights = torch.zeros((M, self.top_k), **f32)
            self.ws_moe = binding.alloc_workspace(
                max(binding.moe_workspace_bytes(H, F, self.experts, m, self.top_k) for m in range(1, M + 1)))
        shapes = [(Q + 2 * KV, H), (H, Q)] + ([] if self.experts else [(2 * F, H), (H, F)])
        self.ws_i8 = binding.alloc_workspace(
            max(binding.i8_workspace_bytes(n, k, m) for n, k in shapes for m in range(1, M + 1)))
        self.ws_head = binding.alloc_workspace(binding.lmhead_workspace_bytes(V, M))
        self.caches = None
        self.tree_mask = self.positions = None

    def layer_weight_bytes(self) -> int:
        L = self.layers[0][0]
        dense = [L.moe] if self.experts else [L.gate_up, L.down]
        return sum(w.nbytes for w in [L.qkv, L.o] + dense) + (0 if L.router is None else 2 * L.router.numel())

    def layer_calls(self, li: int, m: int, copy: int = 0, stream=None) -> list:
        """Layer li's calls at width m, their arguments marshalled."""
        L, H, F, c, s = self.layers[copy][li], self.hidden, self.inter, self.x8, dict(stream=stream)
        norm = dict(eps=self.norm_eps, codes=c[0], scales=c[1], **s)
        # the first layer takes the embedded rows as the residual stream
        x, r = (None, self.x_in) if li == 0 else (self.y_down, self.residual)
        calls = [binding.prepare_add_rmsnorm(x, r, self.residual, L.attn_norm, m, H, **norm),
                 binding.prepare_i8_gemm(L.qkv, *c, m, self.qkv, self.ws_i8, **s)]
        if self.caches:
            calls += self.attention_calls(li, m, stream)
        calls += [binding.prepare_i8_quantize(self.attn_out if self.caches else self.x_o, m, self.qdim, *self.o8, **s),
                  binding.prepare_i8_gemm(L.o, *self.o8, m, self.y_o, self.ws_i8, **s)]
        if self.experts:
            return calls + [
                binding.prepare_add_rmsnorm(self.y_o, self.residual, self.residual, L.mlp_norm, m, H, out=self.normed,
                                            **norm),
                binding.prepare_moe_route(self.normed, L.router, m, self.ids, self.expert_weights, self.ws_moe, **s),
                binding.prepare_moe_mlp(L.moe, *c, m, self.ids, self.expert_weights, self.y_down, self.ws_moe, **s)]
        gate, up = self.gate_up[:, :F], self.gate_up[:, F:]
        return calls + [
            binding.prepare_add_rmsnorm(self.y_o, self.residual, self.residual, L.mlp_norm, m, H, **norm),
            binding.prepare_i8_gemm(L.gate_up, *c, m, self.gate_up, self.ws_i8, **s),
            binding.prepare_silu_mul(gate, up, m, F, codes=self.h8[0], scales=self.h8[1], **s),
            binding.prepare_i8_gemm(L.down, *self.h8, m, self.y_down, self.ws_i8, **s)]

    def final_call(self, m: int, stream=None):
        """The last residual sum and norm: the head's rows."""
        return binding.prepare_add_rmsnorm(self.y_down, self.residual, None, self.final_norm, m, self.hidden,
                                           eps=self.norm_eps, out=self.h, stream=stream)

    def launch_layers(self, m: int, copy: int = 0, stream=None) -> None:
        for call in self.prepare_round(m, copy, stream=stream)[0]:
            call()

    def prepare_round(self, m: int, copy: int, want_logits: bool = False, stream=None):
        layers = [call for li in range(self.n_layers) for call in self.layer_calls(li, m, copy, stream)]
        head = binding.prepare_lmhead(self.heads[copy], self.h, m, self.argmax, self.logits if want_logits else None,
                                      self.ws_head, stream)
        return layers + [self.final_call(m, stream)], head
