"""Python binding of libgpt.so, the B200 GPT pretraining-step library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/gpt.h.  PyTorch provides device
memory and the stream.  If the compiled library is missing the import of
``lib()`` raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgpt.so")

GPT_OK, GPT_EINVAL, GPT_ERANGE, GPT_ETIMEOUT, GPT_ECUDA = 0, -1, -2, -3, -4
KIND_PARAM, KIND_GRAD, KIND_MOM, KIND_ADAM_M, KIND_ADAM_V, KIND_NORMUON_V = 0, 1, 2, 3, 4, 5
REGION_MASTER, REGION_BF16, REGION_GRAD = 0, 1, 2
GROUP_ADAMW, GROUP_MUON = 0, 1
PROF_CATEGORIES = ["qkv_gemm", "proj_gemm", "fc_gemm", "down_gemm", "attn_fwd", "attn_bwd", "logits_gemm",
                   "ce_finish", "lm_dx_gemm", "lm_dw_gemm", "dx_gemm", "dw_gemm", "norm", "qk_bwd", "embed",
                   "ns_gemm", "muon_elem", "adamw", "fp8_quant"]

ABI_FUNCTIONS = [
    "gpt_workspace_size", "gpt_init", "gpt_fwd_bwd", "muon_step", "muon_step_normuon", "muon_step_layers",
    "gpt_block_region", "adamw_step", "gpt_train_step_host", "gpt_num_tensors", "gpt_tensor_info",
    "gpt_get_tensor", "gpt_set_tensor", "gpt_get_row_loss", "gpt_grad_region", "gpt_check",
    "gpt_launch_count", "gpt_profile_enable", "gpt_profile_read", "gpt_destroy", "gpt_last_error",
    "gpt_op_matmul_bf16", "gpt_op_matmul_tf32", "gpt_op_quantize_e4m3", "gpt_op_matmul_fp8",
    "gpt_op_attention_fwd", "gpt_op_attention_bwd", "gpt_op_attention_fwd_ex", "gpt_op_attention_bwd_ex",
    "gpt_op_rmsnorm_fwd", "gpt_op_newton_schulz_scratch", "gpt_op_newton_schulz",
    "gpt_op_newton_schulz_noalloc", "gpt_get_adam_step", "gpt_set_adam_step", "gpt_set_wait_limit",
    "gpt_op_check", "gpt_op_set_wait_limit", "gpt_op_embedding_bwd_scratch", "gpt_op_embedding_bwd",
    "adamw_step_shard", "gpt_tensor_region", "gpt_grad_bucket", "gpt_set_grad_events",
    "gpt_op_attention_plan_bytes", "gpt_op_attention_plan", "gpt_op_attention_packed_fwd",
    "gpt_op_attention_packed_bwd_scratch", "gpt_op_attention_packed_bwd", "gpt_op_policy_loss_scratch",
    "gpt_op_policy_loss", "gpt_op_preference_loss_scratch", "gpt_op_preference_loss",
    "gpt_op_preference_loss_ex", "gpt_op_attention_packed_fwd_ex", "gpt_op_attention_packed_bwd_ex",
]
DTYPE_BF16, DTYPE_FP32 = 0, 1
GRAD_BUCKETS = 6


class GptError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"libgpt error {code}: {msg}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("depth", ctypes.c_int32), ("d_model", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("seq_len", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("mlp_mult", ctypes.c_int32), ("precision", ctypes.c_int32), ("ns_tf32_steps", ctypes.c_int32),
                ("lm_chunk_rows", ctypes.c_int32), ("seed", ctypes.c_uint64), ("short_window", ctypes.c_int32),
                ("window_pattern", ctypes.c_char * 12), ("residual_extras", ctypes.c_int32),
                ("ve_gate_channels", ctypes.c_int32), ("n_kv_head", ctypes.c_int32)]


class HParams(ctypes.Structure):
    _fields_ = [("muon_lr", ctypes.c_float), ("muon_momentum", ctypes.c_float), ("muon_wd", ctypes.c_float),
                ("adam_lr", ctypes.c_float), ("adam_beta1", ctypes.c_float), ("adam_beta2", ctypes.c_float),
                ("adam_eps", ctypes.c_float), ("adam_wd", ctypes.c_float)]


class Heads(ctypes.Structure):
    """gpt_heads: a [tokens, heads, 128] bf16 tensor by pointer and strides."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_LIB = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m gpt_pretraining_step_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        hp, i64 = ctypes.POINTER(Heads), ctypes.c_longlong
        sig = {
            "gpt_workspace_size": (i32, [ctypes.POINTER(Config), ctypes.POINTER(sz), ctypes.POINTER(sz),
                                         ctypes.POINTER(sz)]),
            "gpt_init": (i32, [ctypes.POINTER(Config), vp, vp, vp, vp, ctypes.POINTER(vp)]),
            "gpt_fwd_bwd": (i32, [vp, vp, vp, vp, i32]),
            "muon_step": (i32, [vp, f32, f32, f32]),
            "muon_step_normuon": (i32, [vp, f32, f32, f32, f32]),
            "muon_step_layers": (i32, [vp, f32, f32, f32, f32, i32, i32]),
            "gpt_block_region": (i32, [vp, i32, i32, i32, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "adamw_step": (i32, [vp, f32, f32, f32, f32, f32]),
            "adamw_step_shard": (i32, [vp, f32, f32, f32, f32, f32, i32, i32]),
            "gpt_tensor_region": (i32, [vp, i32, i32, i32, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "gpt_grad_bucket": (i32, [vp, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "gpt_set_grad_events": (i32, [vp, ctypes.POINTER(ctypes.c_void_p), i32]),
            "gpt_train_step_host": (i32, [vp, vp, vp, ctypes.POINTER(HParams), vp]),
            "gpt_num_tensors": (i32, [vp]),
            "gpt_tensor_info": (i32, [vp, i32, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(ctypes.c_int32)]),
            "gpt_get_tensor": (i32, [vp, i32, i32, vp]),
            "gpt_set_tensor": (i32, [vp, i32, i32, vp]),
            "gpt_get_row_loss": (i32, [vp, vp]),
            "gpt_grad_region": (i32, [vp, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "gpt_get_adam_step": (i32, [vp, ctypes.POINTER(ctypes.c_int64)]),
            "gpt_set_adam_step": (i32, [vp, ctypes.c_int64]),
            "gpt_check": (i32, [vp]),
            "gpt_set_wait_limit": (i32, [vp, ctypes.c_longlong]),
            "gpt_op_check": (i32, [vp]),
            "gpt_op_set_wait_limit": (i32, [ctypes.c_longlong]),
            "gpt_launch_count": (ctypes.c_int64, [vp]),
            "gpt_profile_enable": (i32, [vp, ctypes.c_uint32]),
            "gpt_profile_read": (i32, [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]),
            "gpt_destroy": (None, [vp]),
            "gpt_last_error": (ctypes.c_char_p, []),
            "gpt_op_matmul_bf16": (i32, [vp, vp, vp, i32, i32, i32, i32, i32, i32, vp]),
            "gpt_op_matmul_tf32": (i32, [vp, vp, vp, i32, i32, i32, i32, vp]),
            "gpt_op_quantize_e4m3": (i32, [vp, ctypes.c_longlong, vp, vp, vp, vp]),
            "gpt_op_matmul_fp8": (i32, [vp, vp, vp, i32, i32, i32, vp, vp, i32, vp]),
            "gpt_op_attention_fwd": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, vp]),
            "gpt_op_attention_bwd": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]),
            "gpt_op_attention_fwd_ex": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]),
            "gpt_op_attention_bwd_ex": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]),
            "gpt_op_rmsnorm_fwd": (i32, [vp, vp, vp, i32, i32, vp]),
            "gpt_op_embedding_bwd_scratch": (sz, [i32, i32]),
            "gpt_op_embedding_bwd": (i32, [vp, vp, vp, i32, i32, i32, i32, vp, vp]),
            "gpt_op_newton_schulz_scratch": (sz, [i32, i32, i32]),
            "gpt_op_newton_schulz": (i32, [vp, vp, i32, i32, i32, i32, vp, vp]),
            "gpt_op_newton_schulz_noalloc": (i32, [vp, vp, i32, i32, i32, i32, vp]),
            "gpt_op_attention_plan_bytes": (sz, [i32]),
            "gpt_op_attention_plan": (i32, [vp, i32, i32, i32, vp, vp]),
            "gpt_op_attention_packed_bwd_scratch": (sz, [i32, i32]),
            "gpt_op_attention_packed_fwd": (i32, [hp, hp, hp, hp, vp, i32, i32, i32, f32, vp, vp]),
            "gpt_op_attention_packed_bwd": (i32, [hp, hp, hp, hp, vp, hp, hp, hp, hp, i32, i32, i32, f32, vp, vp,
                                                  vp]),
            "gpt_op_attention_packed_fwd_ex": (i32, [hp, hp, hp, hp, vp, i32, i32, i32, f32, vp, i32, vp]),
            "gpt_op_attention_packed_bwd_ex": (i32, [hp, hp, hp, hp, vp, hp, hp, hp, hp, i32, i32, i32, f32, vp, i32,
                                                     vp, vp]),
            "gpt_op_policy_loss_scratch": (sz, [i32]),
            "gpt_op_policy_loss": (i32, [vp, i32, i64, vp, vp, vp, vp, vp, i32, i32, f32, f32, f32, vp, vp, vp, i64,
                                         vp, vp]),
            "gpt_op_preference_loss_scratch": (sz, [i32, i32]),
            "gpt_op_preference_loss": (i32, [vp, i32, i64, vp, vp, i32, vp, i32, i32, f32, f32, vp, vp, vp, vp, vp,
                                             i64, vp, vp]),
            "gpt_op_preference_loss_ex": (i32, [vp, i32, i64, vp, vp, i32, vp, i32, i32, f32, f32, vp, vp, vp, vp, vp,
                                                i64, i32, vp, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(rc):
    if rc != GPT_OK:
        raise GptError(rc, lib().gpt_last_error().decode())
    return rc


def make_config(depth, batch, seq_len, vocab=32768, d_model=0, ns_tf32_steps=-1, lm_chunk_rows=0, seed=0,
                precision=0, window_pattern="", short_window=0, residual_extras=False, ve_gate_channels=0,
                n_kv_head=0):
    return Config(depth=depth, d_model=d_model, vocab=vocab, batch=batch, seq_len=seq_len, head_dim=128,
                  mlp_mult=4, precision=precision, ns_tf32_steps=ns_tf32_steps, lm_chunk_rows=lm_chunk_rows,
                  seed=seed, short_window=short_window, window_pattern=window_pattern.encode("ascii"),
                  residual_extras=int(bool(residual_extras)), ve_gate_channels=int(ve_gate_channels),
                  n_kv_head=int(n_kv_head))


def workspace_size(cfg: Config):
    p, s, a = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gpt_workspace_size(ctypes.byref(cfg), ctypes.byref(p), ctypes.byref(s), ctypes.byref(a)))
    return p.value, s.value, a.value


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class GPTStep:
    """One GPT training-step context on the current CUDA device.

    The three workspace buffers are allocated with torch and owned by this
    object; every computation runs in libgpt's kernels on ``stream``.
    """

    def __init__(self, depth, batch, seq_len, vocab=32768, d_model=0, ns_tf32_steps=-1, lm_chunk_rows=0,
                 seed=0, stream=None, precision=0, window_pattern="", short_window=0, residual_extras=False,
                 ve_gate_channels=0, n_kv_head=0):
        import torch
        self.cfg = make_config(depth, batch, seq_len, vocab, d_model, ns_tf32_steps, lm_chunk_rows, seed, precision,
                               window_pattern, short_window, residual_extras, ve_gate_channels, n_kv_head)
        self.sizes = workspace_size(self.cfg)
        dev = torch.device("cuda", torch.cuda.current_device())
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self.bufs = [torch.empty(max(n, 256), dtype=torch.uint8, device=dev) for n in self.sizes]
        self.loss = torch.zeros(4, dtype=torch.float32, device=dev)
        h = ctypes.c_void_p()
        _check(lib().gpt_init(ctypes.byref(self.cfg), *[_ptr(b) for b in self.bufs], _stream(self.stream),
                              ctypes.byref(h)))
        self.h = h
        self.d_model = self.cfg.d_model or 64 * depth

    def __del__(self):
        h = getattr(self, "h", None)
        if h is not None and _LIB is not None:
            _LIB.gpt_destroy(h)
            self.h = None

    # -- the step
    def fwd_bwd(self, tokens, targets, accumulate=False, loss_out=None):
        out = self.loss if loss_out is None else loss_out
        _check(lib().gpt_fwd_bwd(self.h, _ptr(tokens), _ptr(targets), _ptr(out), int(bool(accumulate))))
        self._join_current_stream()
        return out[0] if loss_out is None else out

    def muon_step(self, lr=0.02, momentum=0.95, weight_decay=0.0):
        _check(lib().muon_step(self.h, lr, momentum, weight_decay))

    def muon_step_normuon(self, lr=0.02, momentum=0.95, weight_decay=0.0, beta2=0.95):
        _check(lib().muon_step_normuon(self.h, lr, momentum, weight_decay, beta2))

    def muon_step_layers(self, l0, l1, lr=0.02, momentum=0.95, weight_decay=0.0, normuon_beta2=-1.0):
        """Muon (or NorMuon with normuon_beta2 >= 0) of layers l0 .. l1-1 only."""
        _check(lib().muon_step_layers(self.h, lr, momentum, weight_decay, normuon_beta2, int(l0), int(l1)))

    def block_region(self, what, kind, l0, l1):
        """Tensor view of block matrix kind (0 q|k|v, 1 attention output, 2 MLP
        up, 3 MLP down) for layers l0 .. l1-1: REGION_MASTER (fp32), REGION_BF16
        (bf16 working copies) or REGION_GRAD (fp32 gradients)."""
        import torch
        off, n = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().gpt_block_region(self.h, int(what), int(kind), int(l0), int(l1), ctypes.byref(off),
                                      ctypes.byref(n)))
        buf = self.bufs[1] if what == REGION_GRAD else self.bufs[0]
        return buf[off.value:off.value + n.value].view(torch.bfloat16 if what == REGION_BF16 else torch.float32)

    def adamw_grad_view(self):
        """fp32 gradients of the token embedding and lm_head (the part of the
        gradient span before the block matrices)."""
        import torch
        off, n = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().gpt_grad_region(self.h, ctypes.byref(off), ctypes.byref(n)))
        first, size = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().gpt_block_region(self.h, REGION_GRAD, 0, 0, 0, ctypes.byref(first), ctypes.byref(size)))
        return self.bufs[1][off.value:first.value].view(torch.float32)

    def adamw_step(self, lr=3e-3, beta1=0.8, beta2=0.95, eps=1e-10, weight_decay=0.0):
        _check(lib().adamw_step(self.h, lr, beta1, beta2, eps, weight_decay))

    def adamw_step_shard(self, part, nparts, lr=3e-3, beta1=0.8, beta2=0.95, eps=1e-10, weight_decay=0.0):
        """AdamW on share `part` of `nparts` of the embedding and lm_head rows
        (the other AdamW tensors whole)."""
        _check(lib().adamw_step_shard(self.h, lr, beta1, beta2, eps, weight_decay, int(part), int(nparts)))

    def tensor_region(self, what, tid, row0, row1):
        """Tensor view of rows row0 .. row1-1 of tensor tid (embedding, lm_head or
        a block matrix): REGION_MASTER, REGION_BF16 or REGION_GRAD."""
        import torch
        off, n = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().gpt_tensor_region(self.h, int(what), int(tid), int(row0), int(row1), ctypes.byref(off),
                                       ctypes.byref(n)))
        buf = self.bufs[1] if what == REGION_GRAD else self.bufs[0]
        return buf[off.value:off.value + n.value].view(torch.bfloat16 if what == REGION_BF16 else torch.float32)

    def grad_bucket(self, i):
        """fp32 view of gradient bucket i (see gpt_grad_bucket)."""
        import torch
        off, n = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().gpt_grad_bucket(self.h, int(i), ctypes.byref(off), ctypes.byref(n)))
        return self.bufs[1][off.value:off.value + n.value].view(torch.float32)

    def set_grad_events(self, events):
        """Register torch.cuda.Event objects: events[i] is recorded on the
        context's stream when gradient bucket i is complete (empty: stop)."""
        self._grad_events = list(events)   # kept alive while registered
        handles = []
        for e in self._grad_events:
            e.record(self.stream)           # creates the event on this device
            handles.append(ctypes.c_void_p(e.cuda_event))
        arr = (ctypes.c_void_p * max(1, len(handles)))(*handles)
        _check(lib().gpt_set_grad_events(self.h, arr, len(handles)))

    def train_step_host(self, tokens_host, targets_host, hp: HParams):
        """Whole step from host int32 arrays (numpy or pinned torch); returns the loss."""
        loss = ctypes.c_float()
        tp = tokens_host.ctypes.data if hasattr(tokens_host, "ctypes") else tokens_host.data_ptr()
        gp = targets_host.ctypes.data if hasattr(targets_host, "ctypes") else targets_host.data_ptr()
        _check(lib().gpt_train_step_host(self.h, ctypes.c_void_p(tp), ctypes.c_void_p(gp), ctypes.byref(hp),
                                         ctypes.byref(loss)))
        return loss.value

    # -- tensors
    def num_tensors(self):
        return lib().gpt_num_tensors(self.h)

    def tensor_info(self, tid):
        r, c, g = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib().gpt_tensor_info(self.h, tid, ctypes.byref(r), ctypes.byref(c), ctypes.byref(g)))
        return r.value, c.value, g.value

    def _shape(self, tid, kind):
        r, c, _ = self.tensor_info(tid)
        return (self.d_model,) if kind == KIND_NORMUON_V else (r, c)

    def get(self, tid, kind=KIND_PARAM):
        """A copy of the tensor, ordered before later work on torch's current
        stream (the copy runs on the context's stream)."""
        import torch
        out = torch.empty(self._shape(tid, kind), dtype=torch.float32, device=self.bufs[0].device)
        _check(lib().gpt_get_tensor(self.h, tid, kind, _ptr(out)))
        self._join_current_stream()
        return out

    def _join_current_stream(self):
        # work queued on the context's stream (a copy into a torch tensor)
        # completes before anything torch's current stream runs next
        import torch
        cur = torch.cuda.current_stream(self.bufs[0].device)
        if cur.cuda_stream != self.stream.cuda_stream:
            cur.wait_stream(self.stream)

    def set(self, tid, value, kind=KIND_PARAM):
        import torch
        shape = self._shape(tid, kind)
        v = torch.as_tensor(value, dtype=torch.float32).to(self.bufs[0].device).contiguous()
        if tuple(v.shape) != shape:
            raise ValueError(f"tensor {tid} has shape {shape}, got {tuple(v.shape)}")
        _check(lib().gpt_set_tensor(self.h, tid, kind, _ptr(v)))
        self.stream.synchronize()

    def grad_view(self):
        """fp32 view of every gradient (one span of the state buffer), e.g. for an all-reduce."""
        import torch
        off, n = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().gpt_grad_region(self.h, ctypes.byref(off), ctypes.byref(n)))
        return self.bufs[1][off.value:off.value + n.value].view(torch.float32)

    def row_loss(self):
        import torch
        out = torch.empty((self.cfg.batch, self.cfg.seq_len), dtype=torch.float32, device=self.bufs[0].device)
        _check(lib().gpt_get_row_loss(self.h, _ptr(out)))
        self._join_current_stream()
        return out

    def check(self):
        return _check(lib().gpt_check(self.h))

    def set_wait_limit(self, cycles):
        """Bound of the kernels' device-side waits in SM cycles (<= 0: the default)."""
        _check(lib().gpt_set_wait_limit(self.h, int(cycles)))

    # -- checkpoint
    def _state_kinds(self, tid):
        _, _, group = self.tensor_info(tid)
        if group == GROUP_MUON:
            return (KIND_PARAM, KIND_MOM, KIND_NORMUON_V)
        return (KIND_PARAM, KIND_ADAM_M, KIND_ADAM_V)

    def state_dict(self):
        """Every tensor's value and optimizer state (host float32 arrays, keyed
        (tensor id, kind)) and the AdamW step count: what a checkpoint needs."""
        step = ctypes.c_int64()
        _check(lib().gpt_get_adam_step(self.h, ctypes.byref(step)))
        tensors = {}
        for tid in range(self.num_tensors()):
            for kind in self._state_kinds(tid):
                tensors[(tid, kind)] = self.get(tid, kind).cpu().numpy()
        return {"tensors": tensors, "adam_step": int(step.value)}

    def load_state_dict(self, state):
        """Restore what state_dict returned (same configuration)."""
        for (tid, kind), value in state["tensors"].items():
            self.set(tid, value, kind)
        _check(lib().gpt_set_adam_step(self.h, int(state["adam_step"])))

    def launch_count(self):
        return lib().gpt_launch_count(self.h)

    def profile_enable(self, categories):
        """Record events around the launches of the named categories (empty = off)."""
        mask = 0
        for c in categories:
            mask |= 1 << PROF_CATEGORIES.index(c)
        _check(lib().gpt_profile_enable(self.h, mask))

    def profile_read(self):
        """{category: (ms, launches)} since the last read (synchronises)."""
        n = len(PROF_CATEGORIES)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        _check(lib().gpt_profile_read(self.h, ms, cnt))
        return {PROF_CATEGORIES[i]: (ms[i], cnt[i]) for i in range(n) if cnt[i]}


# ---------------------------------------------------------------- op level

def op_check(stream=None):
    """Synchronise the stream and raise GptError (GPT_ETIMEOUT) if a bounded
    device wait of an op-level call expired since the last check."""
    return _check(lib().gpt_op_check(_stream(stream)))


def op_set_wait_limit(cycles):
    """Bound of the device-side waits of later op-level calls (<= 0: default)."""
    _check(lib().gpt_op_set_wait_limit(int(cycles)))


def matmul_bf16(A, B, M, N, K, batch=1, a_trans=False, b_trans=False, out=None, stream=None):
    import torch
    C = out if out is not None else torch.empty((batch, M, N), dtype=torch.float32, device=A.device)
    _check(lib().gpt_op_matmul_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, batch, int(a_trans), int(b_trans),
                                    _stream(stream)))
    return C


def matmul_tf32(A, B, M, N, K, b_trans=False, stream=None):
    import torch
    C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check(lib().gpt_op_matmul_tf32(_ptr(A), _ptr(B), _ptr(C), M, N, K, int(b_trans), _stream(stream)))
    return C


def quantize_e4m3(x, stream=None):
    """(q uint8 tensor of e4m3 codes, inv scale tensor) for a bf16 tensor x."""
    import torch
    q = torch.empty(x.numel(), dtype=torch.uint8, device=x.device)
    inv = torch.empty(1, dtype=torch.float32, device=x.device)
    amax = torch.empty(1, dtype=torch.int32, device=x.device)
    _check(lib().gpt_op_quantize_e4m3(_ptr(x), x.numel(), _ptr(q), _ptr(inv), _ptr(amax), _stream(stream)))
    return q.view(x.shape), inv


def matmul_fp8(A, B, M, N, K, inv_a, inv_b, b_trans=False, stream=None):
    import torch
    C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check(lib().gpt_op_matmul_fp8(_ptr(A), _ptr(B), _ptr(C), M, N, K, _ptr(inv_a), _ptr(inv_b), int(b_trans),
                                   _stream(stream)))
    return C


def attention_fwd(q, k, v, window=-1, stream=None):
    """Causal attention; k, v may have fewer heads than q (grouped kv heads);
    window >= 0 limits query t to keys t - window .. t."""
    import torch
    B, H, T, hd = q.shape
    Hkv = k.shape[1]
    o = torch.empty((B, T, H, hd), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    _check(lib().gpt_op_attention_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, T, int(window),
                                         _stream(stream)))
    return o, lse


def attention_bwd(q, k, v, o, lse, dout, window=-1, stream=None):
    import torch
    B, H, T, hd = q.shape
    Hkv = k.shape[1]
    dq = torch.empty((B, H, T, hd), dtype=torch.float32, device=q.device)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    D = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    _check(lib().gpt_op_attention_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(D),
                                         _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, T, int(window), _stream(stream)))
    return dq, dk, dv


# ------------------------------------------------ fine-tuning on packed sequences
#
# A tensor of another type, shape or device than the call takes would be read
# out of range, so these calls check theirs.  They are made once per layer, on
# batches that may be small, where the host's time is the call's: the checks
# compare plain integers, outputs come from an argument's new_empty (a third
# less than torch.empty with its type and device) and the stream as a raw handle.

def _refuse(name, t, want):
    raise GptError(GPT_EINVAL, f"{name} must be {want}; got {t.dtype} {tuple(t.shape)} with strides {t.stride()} "
                               f"on {t.device}")


def _current(torch, name, t):
    """Index of t's device, which has to be the current one (its streams run the call)."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise GptError(GPT_EINVAL, f"{name} is on {t.device}, not on the current CUDA device")
    return dev


def _flat(name, t, dtype, shape, dev):
    """Address of a contiguous tensor argument."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, f"a contiguous {dtype} tensor {shape} on cuda:{dev}")
    return t.data_ptr()


def _heads(name, t, shape, dev, bf16):
    """gpt_heads of a [n, heads, 128] tensor argument."""
    if t.dtype != bf16 or t.shape != shape or t.get_device() != dev:
        _refuse(name, t, f"a bf16 tensor {shape} on cuda:{dev}")
    token, head, one = t.stride()
    if one != 1:
        _refuse(name, t, "a tensor with contiguous rows of 128")
    return Heads(t.data_ptr(), token, head)


def _on(stream, call, *args, **kw):
    """call(*args, **kw) with `stream` as the current one.

    What the call allocates then comes from the pool of the stream that it runs
    on: of another pool it could be a block whose freed tensor that stream still
    uses.  Every tensor of the call is recorded on both streams, so that memory
    dropped on either side is not given out again before the other's queued
    work on it has run.  The order of the two streams' work is the caller's:
    `stream` has to wait for the inputs, the current stream for the results."""
    import torch
    caller = torch.cuda.current_stream()
    if stream.device != caller.device:
        raise GptError(GPT_EINVAL, f"stream is on {stream.device}, the current one on {caller.device}")
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for t in (*args, *kw.values(), *(out or ())):
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
            t.record_stream(caller)
    return out


def _plan_stream(torch, plan):
    """Handle of the current stream.  The buffer of a plan is not the caller's to look after."""
    raw = torch._C._cuda_getCurrentRawStream(plan.device)
    if raw != plan.home:
        plan.buf.record_stream(torch.cuda.current_stream(plan.device))
    return raw


_INT_MAX = 2 ** 31 - 1


@functools.lru_cache(maxsize=256)
def _words(query, *sizes):
    """Size of a plan or scratch buffer in 4-byte words (a pure function of its arguments)."""
    return (max(getattr(lib(), query)(*sizes), 256) + 3) // 4


class AttentionPlan:
    """Masks and work order of one batch of packed sequences (gpt_op_attention_plan)."""

    def __init__(self, cu_seqlens, n_tokens, window=-1, stream=None):
        import torch
        # the C ABI takes 32-bit integers, and binding a larger one drops its upper bits
        self.n_tokens, self.window = int(n_tokens), max(-1, min(int(window), _INT_MAX))
        if not 0 <= self.n_tokens <= _INT_MAX:
            raise GptError(GPT_EINVAL, f"n_tokens must be in [0, 2^30]; got {n_tokens}")
        self.device = _current(torch, "cu_seqlens", cu_seqlens)
        if stream is None:
            self._allocate(torch, cu_seqlens)
        else:
            with torch.cuda.stream(stream):
                self._allocate(torch, cu_seqlens)
        self.update(cu_seqlens, stream)

    def _allocate(self, torch, like):
        self.buf = like.new_empty(_words("gpt_op_attention_plan_bytes", self.n_tokens), dtype=torch.int32)
        self.home = torch._C._cuda_getCurrentRawStream(self.device)   # its memory goes back to this stream

    def update(self, cu_seqlens, stream=None):
        """Plan another batch of the same n_tokens and window into the same buffer."""
        if stream is not None:
            return _on(stream, self.update, cu_seqlens)
        import torch
        _current(torch, "cu_seqlens", cu_seqlens)
        n = cu_seqlens.numel()
        if not 1 <= n <= _INT_MAX:
            _refuse("cu_seqlens", cu_seqlens, "[sequences + 1], up to 2^30 sequences")
        cu = _flat("cu_seqlens", cu_seqlens, torch.int32, (n,), self.device)
        _check(lib().gpt_op_attention_plan(cu, n - 1, self.n_tokens, self.window, self.buf.data_ptr(),
                                           _plan_stream(torch, self)))


def _planned(torch, q, plan):
    """Index of the device of q and its plan."""
    dev = _current(torch, "q", q)
    if plan.device != dev:
        raise GptError(GPT_EINVAL, f"the plan is on cuda:{plan.device}, q on cuda:{dev}")
    return dev


def _head_counts(q, k):
    if q.dim() != 3:
        _refuse("q", q, "[n_tokens, heads, 128]")
    if k.dim() != 3:
        _refuse("k", k, "[n_tokens, kv heads, 128]")
    return q.shape[1], k.shape[1]


def attention_plan(cu_seqlens, n_tokens, window=-1, stream=None):
    """Plan of the sequences cu_seqlens (int32 [n + 1], on the device) packed
    into n_tokens positions, for attention_packed_fwd and _bwd."""
    return AttentionPlan(cu_seqlens, n_tokens, window, stream)


def attention_packed_fwd(q, k, v, plan, scale=0.0, o=None, lse=None, stream=None, clear_past=None):
    """Causal attention of each sequence of the plan.  q [n_tokens, H, 128], k
    and v [n_tokens, Hkv, 128] bf16 with any token and head strides (multiples
    of 8); scale 0 is 1 / sqrt(128).  Returns o [n_tokens, H, 128] and lse
    [H, n_tokens], new unless given.  Rows past the last sequence hold zeros in
    new outputs and keep what they held in given ones; clear_past True or False
    says either of both."""
    if stream is not None:
        return _on(stream, attention_packed_fwd, q, k, v, plan, scale, o, lse, clear_past=clear_past)
    import torch
    clear = (o is None) + 2 * (lse is None) if clear_past is None else 3 * bool(clear_past)   # GPT_CLEAR_*
    n, dev, bf16, f32 = plan.n_tokens, _planned(torch, q, plan), torch.bfloat16, torch.float32
    H, Hkv = _head_counts(q, k)
    rows, kv_rows = (n, H, 128), (n, Hkv, 128)
    hq, hk, hv = (_heads("q", q, rows, dev, bf16), _heads("k", k, kv_rows, dev, bf16),
                  _heads("v", v, kv_rows, dev, bf16))
    if o is None:
        o = q.new_empty(rows)
    if lse is None:
        lse = q.new_empty((H, n), dtype=f32)
    _check(lib().gpt_op_attention_packed_fwd_ex(
        hq, hk, hv, _heads("o", o, rows, dev, bf16), _flat("lse", lse, f32, (H, n), dev), n, H, Hkv, scale,
        plan.buf.data_ptr(), clear, _plan_stream(torch, plan)))
    return o, lse


def attention_packed_bwd(q, k, v, o, lse, dout, plan, scale=0.0, dq=None, dk=None, dv=None, stream=None,
                         clear_past=None):
    """Gradients (bf16, shaped as q, k and v; new unless given) of
    attention_packed_fwd, from its lse and the gradient dout of o (o itself is
    checked but not read: gpt_op_attention_packed_bwd).  Rows past the last
    sequence and clear_past as in the forward."""
    if stream is not None:
        return _on(stream, attention_packed_bwd, q, k, v, o, lse, dout, plan, scale, dq, dk, dv, clear_past=clear_past)
    import torch
    clear = ((dq is None) + 2 * (dk is None) + 4 * (dv is None) if clear_past is None
             else 7 * bool(clear_past))   # GPT_CLEAR_*
    n, dev, bf16, f32 = plan.n_tokens, _planned(torch, q, plan), torch.bfloat16, torch.float32
    H, Hkv = _head_counts(q, k)
    rows, kv_rows = (n, H, 128), (n, Hkv, 128)
    hq, hk, hv = (_heads("q", q, rows, dev, bf16), _heads("k", k, kv_rows, dev, bf16),
                  _heads("v", v, kv_rows, dev, bf16))
    if dq is None:
        dq = q.new_empty(rows)
    if dk is None:
        dk = q.new_empty(kv_rows)
    if dv is None:
        dv = q.new_empty(kv_rows)
    scratch = q.new_empty(_words("gpt_op_attention_packed_bwd_scratch", n, H), dtype=f32)
    _check(lib().gpt_op_attention_packed_bwd_ex(
        hq, hk, hv, _heads("o", o, rows, dev, bf16), _flat("lse", lse, f32, (H, n), dev),
        _heads("dout", dout, rows, dev, bf16), _heads("dq", dq, rows, dev, bf16),
        _heads("dk", dk, kv_rows, dev, bf16), _heads("dv", dv, kv_rows, dev, bf16), n, H, Hkv, scale,
        plan.buf.data_ptr(), clear, scratch.data_ptr(), _plan_stream(torch, plan)))
    return dq, dk, dv


def _rows(name, t, dev):
    """Row stride of a [M, V] tensor argument with contiguous rows."""
    if t.dim() != 2 or t.get_device() != dev:
        _refuse(name, t, f"[M, V] on cuda:{dev}")
    (M, V), (row, one) = t.shape, t.stride()
    if one != 1 and V > 1:
        _refuse(name, t, "[M, V] with contiguous rows")
    return row if M > 1 else max(row, V)


def _loss_rows(torch, logits, grad, dlogits):
    """(M, V, dtype code, row stride, gradient or None, its address and row
    stride, device) of both losses."""
    dev = _current(torch, "logits", logits)
    ld = _rows("logits", logits, dev)
    M, V = logits.shape
    if M > _INT_MAX or V > _INT_MAX:
        _refuse("logits", logits, "[M, V] with M up to 2^30 and V up to 2^24")
    dtype = logits.dtype
    code = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_FP32
    if code == DTYPE_FP32 and dtype != torch.float32:
        _refuse("logits", logits, "bf16 or fp32")
    if not grad:
        return M, V, code, ld, None, None, ld, dev
    ld_d = ld
    if dlogits is None:
        # rows aligned to 16 bytes as the logits' are, without their gaps
        ld_d = V + (ld - V) % (8 if code == DTYPE_BF16 else 4) if M > 1 else V
        dlogits = logits.new_empty((M, V)) if ld_d == V else logits.new_empty_strided((M, V), (ld_d, 1))
    else:
        ld_d = _rows("dlogits", dlogits, dev)
        if dlogits.shape != logits.shape or dlogits.dtype != dtype:
            _refuse("dlogits", dlogits, f"{dtype} {(M, V)}")
    return M, V, code, ld, dlogits, dlogits.data_ptr(), ld_d, dev


def policy_loss(logits, targets, old_logp, advantage, weight, ref_logp=None, kl_coef=0.0, clip_low=0.2,
                clip_high=0.2, grad=True, dlogits=None, stream=None):
    """Clipped policy loss with a KL term and its gradient (gpt_op_policy_loss).

    logits [M, V] bf16 or fp32, targets int32 [M] (-1: not counted); old_logp
    (None: the present ones), advantage, weight and ref_logp (None: no KL
    term) fp32 [M].  Returns (stats [4], logp [M], dlogits): stats are the
    loss and the weighted sums of the clipped surrogate, of the KL estimate
    and of the clipped positions; dlogits (None with grad=False) is new unless
    given, and may be logits itself."""
    if stream is not None:
        return _on(stream, policy_loss, logits, targets, old_logp, advantage, weight, ref_logp, kl_coef, clip_low,
                   clip_high, grad, dlogits)
    import torch
    M, V, code, ld, dlogits, d, ld_d, dev = _loss_rows(torch, logits, grad, dlogits)
    f32, shape = torch.float32, (M,)
    args = (_flat("targets", targets, torch.int32, shape, dev),
            None if old_logp is None else _flat("old_logp", old_logp, f32, shape, dev),
            None if ref_logp is None else _flat("ref_logp", ref_logp, f32, shape, dev),
            _flat("advantage", advantage, f32, shape, dev), _flat("weight", weight, f32, shape, dev))
    stats, logp = weight.new_empty(4), weight.new_empty(M)
    scratch = weight.new_empty(_words("gpt_op_policy_loss_scratch", M))
    _check(lib().gpt_op_policy_loss(
        logits.data_ptr(), code, ld, *args, M, V, clip_low, clip_high, kl_coef, stats.data_ptr(), logp.data_ptr(), d,
        ld_d, scratch.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)))
    return stats, logp, dlogits


def preference_loss(logits, targets, cu_seqlens, ref_logp=None, beta=0.1, label_smoothing=0.0, grad=True,
                    dlogits=None, stream=None, clear_past=None):
    """Preference loss over pairs of packed answers and its gradient
    (gpt_op_preference_loss): sequences 2 i (chosen) and 2 i + 1 (rejected) of
    cu_seqlens int32 [2 pairs + 1].  logits, targets, grad and dlogits as for
    policy_loss; ref_logp fp32 [2 pairs], the reference model's seq_logp.
    Returns (loss [], margin [pairs], seq_logp [2 pairs], logp [M], dlogits).
    Rows past the last sequence: logp and a new dlogits hold zeros there; a
    given dlogits keeps what it held (in place: the logits), or zeros with
    clear_past=True."""
    if stream is not None:
        return _on(stream, preference_loss, logits, targets, cu_seqlens, ref_logp, beta, label_smoothing, grad,
                   dlogits, clear_past=clear_past)
    import torch
    if clear_past is None:
        clear_past = dlogits is None
    M, V, code, ld, dlogits, d, ld_d, dev = _loss_rows(torch, logits, grad, dlogits)
    n, f32, i32 = cu_seqlens.numel() - 1, torch.float32, torch.int32
    if n < 2 or n % 2 or n > _INT_MAX:
        _refuse("cu_seqlens", cu_seqlens, "[2 * pairs + 1]")
    y, cu = _flat("targets", targets, i32, (M,), dev), _flat("cu_seqlens", cu_seqlens, i32, (n + 1,), dev)
    ref = None if ref_logp is None else _flat("ref_logp", ref_logp, f32, (n,), dev)
    loss, margin = logits.new_empty((), dtype=f32), logits.new_empty(n // 2, dtype=f32)
    seq_logp, logp = logits.new_empty(n, dtype=f32), logits.new_empty(M, dtype=f32)
    scratch = targets.new_empty(_words("gpt_op_preference_loss_scratch", M, n // 2))
    _check(lib().gpt_op_preference_loss_ex(
        logits.data_ptr(), code, ld, y, cu, n // 2, ref, M, V, beta, label_smoothing, loss.data_ptr(),
        margin.data_ptr(), seq_logp.data_ptr(), logp.data_ptr(), d, ld_d, bool(clear_past), scratch.data_ptr(),
        torch._C._cuda_getCurrentRawStream(dev)))
    return loss, margin, seq_logp, logp, dlogits


def rmsnorm_fwd(x, stream=None):
    import torch
    M, d = x.shape
    y = torch.empty((M, d), dtype=torch.bfloat16, device=x.device)
    r = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check(lib().gpt_op_rmsnorm_fwd(_ptr(x), _ptr(y), _ptr(r), M, d, _stream(stream)))
    return y, r


def embedding_bwd(tokens, dx, vocab, dwte=None, accumulate=False, stream=None):
    """dwte [vocab, d] (+)= rows of dx [M, d] scattered by token (int32 [M])."""
    import torch
    M, d = dx.shape
    out = torch.zeros((vocab, d), dtype=torch.float32, device=dx.device) if dwte is None else dwte
    scratch = torch.empty(max(lib().gpt_op_embedding_bwd_scratch(M, d), 256), dtype=torch.uint8, device=dx.device)
    _check(lib().gpt_op_embedding_bwd(_ptr(tokens), _ptr(dx), _ptr(out), M, d, vocab, int(bool(accumulate)),
                                      _ptr(scratch), _stream(stream)))
    return out


def newton_schulz(G, tf32_steps=-1, stream=None):
    import torch
    batch, rows, cols = G.shape
    X = torch.empty_like(G)
    n = lib().gpt_op_newton_schulz_scratch(batch, rows, cols)
    scratch = torch.empty(n, dtype=torch.uint8, device=G.device)
    _check(lib().gpt_op_newton_schulz(_ptr(G), _ptr(X), batch, rows, cols, tf32_steps, _ptr(scratch),
                                      _stream(stream)))
    return X


def newton_schulz_noalloc(G, tf32_steps=-1, X=None, stream=None):
    """Newton-Schulz through the entry point that allocates no device memory.

    The library keeps the scratch in its own fixed device array (at most
    batch * rows * cols = 262144 elements); only the output is caller memory.
    Calls that overlap on the GPU share that array and must not run
    concurrently.
    """
    import torch
    batch, rows, cols = G.shape
    X = torch.empty_like(G) if X is None else X
    _check(lib().gpt_op_newton_schulz_noalloc(_ptr(G), _ptr(X), batch, rows, cols, tf32_steps, _stream(stream)))
    return X
