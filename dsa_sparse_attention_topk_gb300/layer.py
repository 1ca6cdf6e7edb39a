"""One DSA attention layer's decode state: the two paged caches and the calls of a decode
step, on one CUDA device.  Plumbing only -- torch allocates the memory and every
computation is a call into the C ABI.
"""

import torch

from . import (V_DIM, alloc_k_cache, alloc_kv_cache, attn_mass, attn_mass_workspace_size, quant_kv_mxfp8, quant_kv_fp8,
               decode_step, evict_compact, evict_select, indexer_topk, norm_rope, norm_rope_quant_kv, prefix_attn, rope,
               rope_quant_kv, sparse_attn, sparse_attn_mass, sparse_attn_workspace_size)


class DsaDecodeLayer:
    """Paged MXFP8 indexer K-cache + paged FP8 latent cache of ``num_pages`` 64-token pages.

    A decode step writes the step's new tokens into both caches, runs the fused indexer +
    Top-K, then sparse attention over the selected entries.

    rope  None: queries, keys and latent rows come with their positions already in them.
          (turns, amplitude), as rope_turns(64) returns them: they come without, and every call turns them:
          the 64 dims from index_offset of indexer queries and keys in index_layout, the last
          64 of attention queries and latent rows in latent_layout.
    norm  with rope: the norms of norm_rope_quant_kv that indexer keys and latent rows get before they are turned, a dict
          of its k_weight, k_bias, kv_weight, k_norm and eps, each as there if left out.  None: they come normed.
    index_norm  with rope: the norm of norm_rope that the heads of indexer queries get before they are turned, a dict of its
          weight, bias, norm, norm_dim and eps.  None: they come normed.

    What the cache's positions are worth to the attention can be added up (``mass`` of decode, step and attend_prefix,
    int64 [n_seq, max_ctx], zero at first, as wide as the longest sequence) and the least used ones given up (``evict``).  The records that
    stay move to the first positions of their sequence and keep the turns they have: from then on rope_pos, the
    positions to turn to, differ from q_pos, the places in the cache.
    """

    def __init__(self, num_pages, h_i, h_s, topk, sm_scale, device="cuda", rope=None, index_offset=0,
                 index_layout="half", latent_layout="interleaved", norm=None, index_norm=None):
        self.device = torch.device(device)
        self.rope, self.index_offset = rope, index_offset
        self.index_layout, self.latent_layout = index_layout, latent_layout
        for name, given, known in (("norm", norm, ("k_weight", "k_bias", "kv_weight", "k_norm", "eps")),
                                   ("index_norm", index_norm, ("weight", "bias", "norm", "norm_dim", "eps"))):
            if given is None:
                continue
            if rope is None:
                raise ValueError(f"DsaDecodeLayer: {name} goes with rope")
            if set(given) - set(known):
                raise ValueError(f"DsaDecodeLayer: {name} knows {', '.join(known)}")
        self.norm, self.index_norm = norm, index_norm
        self.num_pages = int(num_pages)
        self.h_i, self.h_s, self.topk, self.sm_scale = h_i, h_s, topk, float(sm_scale)
        self.k_cache = alloc_k_cache(num_pages, self.device)
        self.kv_cache = alloc_kv_cache(num_pages, self.device)
        self._bufs = {}

    def write(self, k, kv, slot_mapping, pos=None):
        """Quantise and store new tokens: k bf16 [n, 128], kv bf16 [n, 576], slots int64 [n];
        with rope also their positions, int32 [n]."""
        if self.rope is None:
            quant_kv_mxfp8(k, slot_mapping, self.k_cache)
            quant_kv_fp8(kv, slot_mapping, self.kv_cache)
            return
        if pos is None:
            raise ValueError("write: a layer with rope needs the tokens' positions")
        turns, amplitude = self.rope
        if self.norm is not None:
            norm_rope_quant_kv(k, kv, pos, slot_mapping, self.k_cache, self.kv_cache, turns, amplitude=amplitude,
                               k_offset=self.index_offset, k_layout=self.index_layout, kv_layout=self.latent_layout,
                               **self.norm)
            return
        rope_quant_kv(k, kv, pos, slot_mapping, self.k_cache, self.kv_cache, turns, amplitude=amplitude,
                      k_offset=self.index_offset, k_layout=self.index_layout, kv_layout=self.latent_layout)

    def _turn_index(self, q, pos, out=None):
        turns, amplitude = self.rope
        if self.index_norm is not None:
            return norm_rope(q, pos, turns, offset=self.index_offset, layout=self.index_layout, amplitude=amplitude, out=out,
                             **self.index_norm)
        return rope(q, pos, turns, offset=self.index_offset, layout=self.index_layout, amplitude=amplitude, out=out)

    def _turn_latent(self, q, pos, out=None):
        turns, amplitude = self.rope
        return rope(q, pos, turns, offset=V_DIM, layout=self.latent_layout, amplitude=amplitude, out=out)

    def _buffers(self, n_q):
        b = self._bufs.get(n_q)
        if b is None:
            dev = self.device
            b = {
                "idx": torch.empty(n_q, self.topk, dtype=torch.int32, device=dev),
                "out": torch.empty(n_q, self.h_s, 512, dtype=torch.bfloat16, device=dev),
                "lse": torch.empty(n_q, self.h_s, dtype=torch.float32, device=dev),
                "mass_ws": {},
            }
            ws = sparse_attn_workspace_size(n_q, self.h_s, self.topk)
            b["ws"] = torch.empty(max(ws, 1), dtype=torch.uint8, device=dev) if ws else None
            if self.rope is not None:  # the turned queries
                b["q_idx"] = torch.empty(n_q, self.h_i, 128, dtype=torch.bfloat16, device=dev)
                b["q_sfa"] = torch.empty(n_q, self.h_s, 576, dtype=torch.bfloat16, device=dev)
            self._bufs[n_q] = b
        return b

    def _mass_ws(self, n_q, n_seq, b):
        """The workspace of a step's weights, one of the buffers b.  Sequences count where there are more of them than rows:
        then by powers of two, each with a workspace that stays, for a recorded step may hold it."""
        most = n_q if n_seq <= n_q else min(1 << (n_seq - 1).bit_length(), max(n_seq, 65536))
        ws = b["mass_ws"].get(most)
        if ws is None:
            ws = torch.empty(attn_mass_workspace_size(n_q, self.h_s, most), dtype=torch.uint8, device=self.device)
            b["mass_ws"][most] = ws
        return ws

    def _weigh(self, mass, q_sfa, page_table, seq_lens, q_seq, b):
        """Add the weights of the entries that a step selected."""
        if "weights" not in b:
            b["weights"] = torch.empty(b["idx"].shape, dtype=torch.float32, device=self.device)
        sparse_attn_mass(q_sfa, self.kv_cache, page_table, seq_lens, q_seq, b["idx"], b["lse"], self.sm_scale, mass=mass,
                         out=b["weights"], workspace=self._mass_ws(q_sfa.shape[0], seq_lens.shape[0], b))

    def decode(self, q_idx, w, q_sfa, page_table, seq_lens, q_seq, q_pos, max_ctx, q_group=1, rope_pos=None, mass=None):
        """Indexer + Top-K + SFA for n_q query rows.  Returns (out bf16 [n_q, h_s, 512],
        lse fp32 [n_q, h_s], idx int32 [n_q, topk]); the tensors are reused by the next
        call with the same n_q.  rope_pos (int32 [n_q]) are the positions that queries are turned to, q_pos if left
        out; to mass the weights of the selected positions are added."""
        n_q = q_idx.shape[0]
        b = self._buffers(n_q)
        if self.rope is not None:
            rope_pos = q_pos if rope_pos is None else rope_pos
            q_idx = self._turn_index(q_idx, rope_pos, b["q_idx"])
            q_sfa = self._turn_latent(q_sfa, rope_pos, b["q_sfa"])
        indexer_topk(q_idx, w, self.k_cache, page_table, seq_lens, q_seq, q_pos, self.topk, max_ctx,
                     q_group=q_group, out_idx=b["idx"])
        sparse_attn(q_sfa, self.kv_cache, page_table, seq_lens, q_seq, b["idx"], self.sm_scale,
                    out=b["out"], out_lse=b["lse"], workspace=b["ws"])
        if mass is not None:
            self._weigh(mass, q_sfa, page_table, seq_lens, q_seq, b)
        return b["out"], b["lse"], b["idx"]

    def attend_prefix(self, q_sfa, prefix_pages, prefix_len, page_table, seq_lens, q_seq, q_pos, max_ctx, rope_pos=None,
                      mass=None):
        """Dense attention of n_q query rows whose sequences share their first prefix_len
        positions (prefix_pages, read once for all rows), each row then over its own ones up to
        q_pos.  Returns (out bf16 [n_q, h_s, 512], lse fp32 [n_q, h_s]), new tensors each call.  rope_pos as for decode;
        to mass the weights of every position seen are added, for which page_table names the shared pages too."""
        if mass is not None and page_table is None:
            raise ValueError("attend_prefix: mass needs a page_table")
        if self.rope is not None:
            q_sfa = self._turn_latent(q_sfa, q_pos if rope_pos is None else rope_pos)
        lse = torch.empty(q_sfa.shape[0], self.h_s, dtype=torch.float32, device=self.device)
        out = prefix_attn(q_sfa, self.kv_cache, prefix_pages, prefix_len, page_table, seq_lens, q_seq, q_pos, max_ctx,
                          self.sm_scale, out_lse=lse)
        if mass is not None:
            attn_mass(q_sfa, self.kv_cache, page_table, seq_lens, q_seq, q_pos, lse, max_ctx, self.sm_scale, mass=mass)
        return out

    def evict(self, mass, page_table, seq_lens, budget, sinks=0, recent=0, dst_table=None):
        """Keep budget positions of each sequence: the first sinks, the last recent and those of the largest mass between
        (evict_select); move their records to the sequence's first positions, in place or to the pages of dst_table
        (evict_compact), and their mass with them; the rest of mass becomes 0.  Returns (kept int32 [n_seq, budget]: the
        positions that stayed, -1 behind the last; new_lens int32 [n_seq]).  Pages behind the new lengths are free.
        In place, sequences must not share pages that are written."""
        kept, new_lens, kept_mass = evict_select(mass, seq_lens, budget, sinks=sinks, recent=recent)
        evict_compact(kept, page_table, self.k_cache, self.kv_cache, dst_table)
        n = min(budget, mass.shape[1])  # (what would lie further is empty)
        mass[:, :n].copy_(kept_mass[:, :n])
        mass[:, n:].zero_()
        return kept, new_lens

    def step(self, k_new, kv_new, slots_new, q_idx, w, q_sfa, page_table, seq_lens, q_seq, q_pos,
             max_ctx, q_group=1, pos_new=None, rope_pos=None, mass=None):
        """Write this step's tokens into both caches, then decode: one library call
        (dsa_decode_step).  With one new token per query row the indexer kernel writes the
        tokens itself, each before it loads the page that holds it, and SFA follows it on
        the current stream with programmatic dependent launch; otherwise a writer kernel
        runs first and the indexer reads its other inputs while the writer runs.

        With rope the new tokens are turned and written by one kernel, the queries turned by
        two more, before that call.  pos_new (int32) are the new tokens' positions; left out,
        token i is query row i's own and is turned with it.  rope_pos and mass as for decode.
        """
        n_q = q_idx.shape[0]
        b = self._buffers(n_q)
        if self.rope is not None:
            rope_pos = q_pos if rope_pos is None else rope_pos
            if pos_new is None:
                if k_new.shape[0] != n_q:
                    raise ValueError("step: pos_new is needed unless there is one new token per query row")
                pos_new = rope_pos
            self.write(k_new, kv_new, slots_new, pos_new)
            q_idx = self._turn_index(q_idx, rope_pos, b["q_idx"])
            q_sfa = self._turn_latent(q_sfa, rope_pos, b["q_sfa"])
            k_new, kv_new, slots_new = k_new[:0], kv_new[:0], slots_new[:0]
        decode_step(k_new, kv_new, slots_new, self.k_cache, self.kv_cache, q_idx, w, q_sfa, page_table,
                    seq_lens, q_seq, q_pos, self.topk, max_ctx, self.sm_scale, q_group=q_group,
                    out_idx=b["idx"], out=b["out"], out_lse=b["lse"], workspace=b["ws"],
                    stream=torch.cuda.current_stream(self.device))
        if mass is not None:
            self._weigh(mass, q_sfa, page_table, seq_lens, q_seq, b)
        return b["out"], b["lse"], b["idx"]

    def capture_step(self, inputs, max_ctx, q_group=1, stage=None, result=None):
        """Record one decode step (``step`` on the tensors of ``inputs``) into a CUDA graph
        and return a function that replays it on the current stream.

        inputs  dict with the ``step`` arguments k_new, kv_new, slots_new, q_idx, w, q_sfa,
                page_table, seq_lens, q_seq, q_pos (and pos_new where step needs it, rope_pos,
                mass): device tensors that stay in place; a replay reads whatever they hold
                then and adds to mass.  Recording itself runs the step once, without mass.
        stage   optional (pinned host tensor, device tensor) pair copied host -> device at
                the start of every replay (the step's inputs staged in one buffer).
        result  optional pinned host tensor [n_q, h_s, 512] bf16 that receives the output at
                the end of every replay.

        The graph holds the launches of one ``dsa_decode_step`` with their programmatic
        dependencies, so a replay costs one graph launch instead of the host work of each
        call.  The returned function also exposes ``out``, ``lse`` and ``idx``, the device
        tensors the replays write.
        """
        keys = ("k_new", "kv_new", "slots_new", "q_idx", "w", "q_sfa", "page_table", "seq_lens", "q_seq", "q_pos")
        args = [inputs[k] for k in keys]
        pos_new, rope_pos, mass = (inputs.get(k) for k in ("pos_new", "rope_pos", "mass"))
        # one eager step first: per-device queries, kernel attributes and the output buffers
        # are set up outside the capture
        side = torch.cuda.Stream(self.device)
        side.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(side):
            if stage is not None:
                stage[1].copy_(stage[0], non_blocking=True)
            self.step(*args, max_ctx, q_group, pos_new, rope_pos, None if mass is None else torch.zeros_like(mass))
        torch.cuda.current_stream(self.device).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        # (relaxed: the library's host-side queries during the capture are not stream work)
        with torch.cuda.graph(graph, capture_error_mode="relaxed"):
            if stage is not None:
                stage[1].copy_(stage[0], non_blocking=True)
            out, lse, idx = self.step(*args, max_ctx, q_group, pos_new, rope_pos, mass)
            if result is not None:
                result.copy_(out, non_blocking=True)

        def replay():
            graph.replay()

        replay.out, replay.lse, replay.idx, replay.graph = out, lse, idx, graph
        return replay
