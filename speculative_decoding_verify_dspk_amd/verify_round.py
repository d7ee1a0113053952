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
