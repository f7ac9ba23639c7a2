"""ctypes binding of libgpt.so (include/gpt.h, include/gpt_testing.h).

Argument marshalling only: every step of the training step runs in the CUDA
library.  PyTorch provides device memory (the workspace) and the stream.
Loading fails loudly when the library has not been built.
"""

from __future__ import annotations

import ctypes as C
import os
import re
from typing import Dict, List, Optional, Tuple

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgpt.so")
HEADERS = [os.path.join(os.path.dirname(_PKG), "include", h) for h in ("gpt.h", "gpt_testing.h")]

GPT_ABI_VERSION = 2
GPT_PREC_FP32, GPT_PREC_BF16 = 0, 1
GPT_VARIANT_GPT2, GPT_VARIANT_MICRO = 0, 1
GPT_TOK_I32, GPT_TOK_U16 = 0, 1
GPT_PARAM, GPT_GRAD, GPT_ADAM_M, GPT_ADAM_V = 0, 1, 2, 3
GPT_PATH_GEMM_TC, GPT_PATH_ATTN_TC = 1, 2
STATUS = ["GPT_OK", "GPT_ERR_INVALID_ARG", "GPT_ERR_CONFIG", "GPT_ERR_WORKSPACE_TOO_SMALL", "GPT_ERR_CUDA",
          "GPT_ERR_TOKEN_RANGE", "GPT_ERR_NONFINITE", "GPT_ERR_STATE", "GPT_ERR_UNSUPPORTED", "GPT_ERR_TIMEOUT"]
FLAG_TOKEN, FLAG_LOSS, FLAG_NORM, FLAG_TIMEOUT = 1, 2, 4, 8
FLAG_BLOCK_RANGE, FLAG_CACHE_FULL, FLAG_ROW_RANGE = 16, 32, 64


class GptConfig(C.Structure):
    _fields_ = [
        ("abi_version", C.c_uint32), ("vocab_size", C.c_int32), ("padded_vocab", C.c_int32),
        ("n_layer", C.c_int32), ("n_head", C.c_int32), ("n_embd", C.c_int32), ("block_size", C.c_int32),
        ("batch_size", C.c_int32), ("grad_accum", C.c_int32), ("precision", C.c_int32), ("variant", C.c_int32),
        ("token_dtype", C.c_int32), ("dropout", C.c_float), ("beta1", C.c_float),
        ("beta2", C.c_float), ("eps", C.c_float), ("weight_decay", C.c_float), ("grad_clip", C.c_float),
        ("decay_1d", C.c_int32), ("recompute", C.c_int32), ("dropout_seed", C.c_uint64),
        ("init_std", C.c_double), ("zero_world", C.c_int32), ("zero_rank", C.c_int32),
    ]


class Kv8CacheStruct(C.Structure):  # gpt_kv8_cache
    _fields_ = [
        ("n_seq", C.c_int32), ("n_head_kv", C.c_int32), ("head_dim", C.c_int32), ("block_tokens", C.c_int32),
        ("n_blocks", C.c_int32), ("max_blocks", C.c_int32), ("d_k", C.c_void_p), ("d_v", C.c_void_p),
        ("d_k_scale", C.c_void_p), ("d_v_scale", C.c_void_p), ("d_weight", C.c_void_p), ("d_table", C.c_void_p),
        ("d_len", C.c_void_p), ("d_flags", C.c_void_p),
    ]


class GptError(RuntimeError):
    def __init__(self, status: int, msg: str):
        self.status = status
        self.name = STATUS[status] if 0 <= status < len(STATUS) else str(status)
        super().__init__(f"{self.name}: {msg}")


_lib = None
P, I32, I64, U32, U64, F32, SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_uint32, C.c_uint64, C.c_float, C.c_size_t
_PROTOS = {
    "gpt_param_count": (SZ, [P]),
    "gpt_config_kernel_paths": (I32, [P, P]),
    "gpt_workspace_bytes": (I32, [P, P]),
    "gpt_grad_buckets": (I32, [P, I32, P, P, P, P]),
    "gpt_grad_arena": (I32, [P, P, P]),
    "gpt_zero1_shard": (I32, [P, I32, I32, P, P, P]),
    "gpt_state_arenas": (I32, [P, P, P, P, P, P, P, P, P]),
    "gpt_grad_sumsq_shard": (I32, [P, I64, I64, P]),
    "gpt_clip_adamw_shard": (I32, [P, F32, I32, I64, I64, F32, P, I32, P]),
    "gpt_train_step_accumulate": (I32, [P, P, U64, U64, I32, P]),
    "gpt_stream_wait_bucket": (I32, [P, I32, P]),
    "gpt_step_loss": (I32, [P, P]),
    "gpt_train_step_host_accumulate": (I32, [P, P, P, I32, P]),
    "gpt_lr_cosine": (F32, [F32, I32, I32, I32]),
    "gpt_lr_linear": (F32, [F32, I32, I32]),
    "gpt_create": (I32, [P, U64, P, SZ, P, P]),
    "gpt_destroy": (None, [P]),
    "gpt_set_stream": (I32, [P, P]),
    "gpt_forward_loss": (I32, [P, P, P, P]),
    "gpt_backward": (I32, [P]),
    "gpt_clip_adamw_step": (I32, [P, F32, I32, P]),
    "gpt_train_step": (I32, [P, P, U64, U64, F32, I32, P, P]),
    "gpt_train_step_host": (I32, [P, P, P, F32, I32, P, P]),
    "gpt_gather_batch": (I32, [P, P, U64, U64, I32, I32, P, P]),
    "gpt_set_dropout_cursor": (I32, [P, I32, I32]),
    "gpt_set_graphs": (I32, [P, I32]),
    "gpt_eval_loss": (I32, [P, P, U64, U64, I32, P]),
    "gpt_sample": (I32, [P, I32, I32, I32, I64, F32, I32, F32, P, P, P]),
    "gpt_generate": (I32, [P, P, I32, I32, F32, I32, F32, P, P]),
    "gpt_generate_kv8": (I32, [P, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, P]),
    "gpt_sample_rows": (I32, [P, I32, I32, I32, I64, P, P, P, P, P, P, P, P]),
    "gpt_kv8_append": (I32, [P, P, I32, I32, I32, P, I64, P, I64, P]),
    "gpt_kv8_attention": (I32, [P, P, I32, I32, I32, I32, P, I64, F32, I32, P, I64, P, P]),
    "gpt_kv8_accumulate": (I32, [P, P, I32, I32, I32, I32, P, I64, F32, I32, P, P]),
    "gpt_kv8_evict": (I32, [P, P, I32, I32, I32, P, P]),
    "gpt_kv8_advance": (I32, [P, P, I32, I32, I32, P]),
    "gpt_lora_workspace_bytes": (I32, [P, I32, I32, P]),
    "gpt_lora_attach": (I32, [P, I32, F32, I32, P, P, SZ]),
    "gpt_lora_detach": (I32, [P]),
    "gpt_lora_read": (I32, [P, I32, P, SZ]),
    "gpt_lora_write": (I32, [P, P, SZ]),
    "gpt_num_tensors": (I32, [P, P]),
    "gpt_tensor_info": (I32, [P, I32, P, P]),
    "gpt_get_tensor": (I32, [P, I32, I32, P]),
    "gpt_set_tensor": (I32, [P, I32, I32, P]),
    "gpt_get_logits": (I32, [P, P]),
    "gpt_get_argmax": (I32, [P, P]),
    "gpt_argmax_rows": (I32, [P, P, I32, I32, P]),
    "gpt_get_lse": (I32, [P, P]),
    "gpt_get_embed_routing": (I32, [P, P, P, P]),
    "gpt_dropout_mask": (I32, [P, I64, I32, I32, I64, P]),
    "gpt_state_floats": (SZ, [P]),
    "gpt_get_state": (I32, [P, P, P, P]),
    "gpt_set_state": (I32, [P, P, P, P]),
    "gpt_read_flags": (I32, [P, P]),
    "gpt_clear_flags": (I32, [P]),
    "gpt_enable_timing": (I32, [P, I32]),
    "gpt_kernel_times": (I32, [P, I32, P, P, P, P]),
    "gpt_launch_count": (U64, [P]),
    "gpt_last_error": (C.c_char_p, [P]),
    "gpt_status_string": (C.c_char_p, [I32]),
    "gpt_test_gemm": (I32, [I32, I32, I32, I32, P, I64, I32, P, I64, I32, I32, I32, P, P, I32, P, P, P, P, I32, P,
                            P, P, P]),
    "gpt_test_attention": (I32, [I32, I32, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, F32, U64, U64, I32, P, P]),
    "gpt_test_wait_timeout": (I32, [U64, P, P, P]),
    "gpt_gemm_dw_accumulate_noalloc": (I32, [I32, I32, I32, P, I64, P, I64, P, I32, P]),
}


def lib() -> C.CDLL:
    """The loaded CUDA library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m gpt_decoder_lm_b200.build`")
        l = C.CDLL(LIB_PATH)
        for name, (res, args) in _PROTOS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def declared_symbols() -> List[str]:
    """Function names declared in include/*.h."""
    out = []
    for h in HEADERS:
        txt = open(h).read()
        txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
        out += re.findall(r"\b(gpt_[a-z0-9_]+)\s*\(", txt)
    return sorted(set(out))


def _check(st: int, model=None, what: str = ""):
    if st != 0:
        msg = lib().gpt_last_error(model).decode() if model else ""
        raise GptError(st, f"{what} {msg}".strip())


def _ptr(a) -> int:
    """Device or host address of a torch tensor / numpy array (None -> 0)."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        assert a.flags["C_CONTIGUOUS"]
        return a.ctypes.data
    return a.data_ptr()


def make_config(w, **over) -> GptConfig:
    """gpt_config from a workloads.Workload (keyword overrides allowed)."""
    d = dict(vocab_size=w.vocab_size, n_layer=w.n_layer, n_head=w.n_head, n_embd=w.n_embd,
             block_size=w.block_size, batch_size=w.batch_size, grad_accum=w.grad_accum,
             precision=GPT_PREC_BF16 if w.precision == "bf16" else GPT_PREC_FP32,
             variant=GPT_VARIANT_MICRO if w.variant == "micro" else GPT_VARIANT_GPT2,
             token_dtype=GPT_TOK_U16 if w.token_dtype == "uint16" else GPT_TOK_I32,
             init_std=w.init_std, dropout=w.dropout, beta1=w.beta1, beta2=w.beta2, eps=w.eps,
             weight_decay=w.weight_decay, grad_clip=w.grad_clip, decay_1d=0, dropout_seed=w.dropout_seed,
             padded_vocab=0)
    d.update(over)
    c = GptConfig()
    c.abi_version = GPT_ABI_VERSION
    for k, v in d.items():
        setattr(c, k, v)
    return c


def grad_buckets(cfg: GptConfig):
    """The gradient exchange plan: [(offset, count, bucket)] in the order the
    backward finalises the buckets."""
    n = C.c_int32(0)
    _check(lib().gpt_grad_buckets(C.byref(cfg), 0, None, None, None, C.byref(n)), None, "grad_buckets")
    off = (C.c_int64 * n.value)()
    cnt = (C.c_int64 * n.value)()
    bkt = (C.c_int32 * n.value)()
    _check(lib().gpt_grad_buckets(C.byref(cfg), n.value, off, cnt, bkt, C.byref(n)), None, "grad_buckets")
    return [(int(off[i]), int(cnt[i]), int(bkt[i])) for i in range(n.value)]


NORM_PARTIALS = 592  # GPT_NORM_PARTIALS


def zero1_shard(cfg: GptConfig, world: int, rank: int):
    """(offset, count, stride) of optimiser shard `rank` of `world`."""
    off, cnt, stride = C.c_int64(), C.c_int64(), C.c_int64()
    _check(lib().gpt_zero1_shard(C.byref(cfg), world, rank, C.byref(off), C.byref(cnt), C.byref(stride)), None,
           "zero1_shard")
    return int(off.value), int(cnt.value), int(stride.value)


def kernel_paths(cfg: GptConfig) -> int:
    """GPT_PATH_* bits: which kernels a model with this config runs."""
    n = C.c_uint32(0)
    _check(lib().gpt_config_kernel_paths(C.byref(cfg), C.byref(n)), None, "config_kernel_paths")
    return int(n.value)


def param_count(cfg: GptConfig) -> int:
    return int(lib().gpt_param_count(C.byref(cfg)))


def workspace_bytes(cfg: GptConfig) -> int:
    n = C.c_size_t(0)
    _check(lib().gpt_workspace_bytes(C.byref(cfg), C.byref(n)), None, "workspace_bytes")
    return int(n.value)


def lr_cosine(lr, it, warmup, max_iters) -> float:
    return float(lib().gpt_lr_cosine(lr, it, warmup, max_iters))


def lr_linear(lr, it, max_iters) -> float:
    return float(lib().gpt_lr_linear(lr, it, max_iters))


class Model:
    """One model in a torch-allocated device workspace, on torch's current stream."""

    def __init__(self, cfg: GptConfig, seed: int, device=None, stream=None, workspace=None):
        import torch
        self.cfg = cfg
        self.device = torch.device(device or "cuda")
        nbytes = workspace_bytes(cfg)
        self.ws = workspace if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.stream = stream or torch.cuda.current_stream(self.device)
        h = C.c_void_p()
        st = lib().gpt_create(C.byref(cfg), seed, self.ws.data_ptr(), self.ws.numel(), self.stream.cuda_stream,
                              C.byref(h))
        _check(st, None, "gpt_create")
        self.h = h
        self.M = cfg.batch_size * cfg.block_size

    def close(self):
        h = getattr(self, "h", None)
        if h:
            self.h = None
            f = globals().get("lib")  # None while the interpreter shuts down
            if f is not None:
                f().gpt_destroy(h)

    __del__ = close

    # -- step
    def forward_loss(self, idx, tgt, sync: bool = True) -> Optional[float]:
        out = C.c_float()
        _check(lib().gpt_forward_loss(self.h, _ptr(idx), _ptr(tgt), C.byref(out) if sync else None), self.h,
               "forward_loss")
        return float(out.value) if sync else None

    def backward(self):
        _check(lib().gpt_backward(self.h), self.h, "backward")

    def clip_adamw_step(self, lr: float, step: int, sync: bool = True) -> Optional[float]:
        out = C.c_float()
        _check(lib().gpt_clip_adamw_step(self.h, lr, step, C.byref(out) if sync else None), self.h, "clip_adamw")
        return float(out.value) if sync else None

    def train_step(self, stream_tokens, data_seed: int, lr: float, step: int, sync: bool = True):
        loss, norm = C.c_float(), C.c_float()
        _check(lib().gpt_train_step(self.h, _ptr(stream_tokens), stream_tokens.numel(), data_seed, lr, step,
                                    C.byref(loss) if sync else None, C.byref(norm) if sync else None), self.h,
               "train_step")
        return (float(loss.value), float(norm.value)) if sync else None

    def train_step_host(self, h_idx, h_tgt, lr: float, step: int):
        loss, norm = C.c_float(), C.c_float()
        _check(lib().gpt_train_step_host(self.h, _ptr(h_idx), _ptr(h_tgt), lr, step, C.byref(loss), C.byref(norm)),
               self.h, "train_step_host")
        return float(loss.value), float(norm.value)

    def train_step_accumulate(self, stream_tokens, data_seed: int, step: int, sync: bool = False):
        loss = C.c_float()
        _check(lib().gpt_train_step_accumulate(self.h, _ptr(stream_tokens), stream_tokens.numel(), data_seed, step,
                                               C.byref(loss) if sync else None), self.h, "train_step_accumulate")
        return float(loss.value) if sync else None

    def train_step_host_accumulate(self, h_idx, h_tgt, step: int, sync: bool = False):
        loss = C.c_float()
        _check(lib().gpt_train_step_host_accumulate(self.h, _ptr(h_idx), _ptr(h_tgt), step,
                                                    C.byref(loss) if sync else None), self.h,
               "train_step_host_accumulate")
        return float(loss.value) if sync else None

    def step_loss(self) -> float:
        out = C.c_float()
        _check(lib().gpt_step_loss(self.h, C.byref(out)), self.h, "step_loss")
        return float(out.value)

    def stream_wait_bucket(self, bucket: int, stream):
        _check(lib().gpt_stream_wait_bucket(self.h, bucket, stream.cuda_stream), self.h, "stream_wait_bucket")

    def grad_arena(self):
        """The fp32 gradient arena as a torch tensor view of the workspace."""
        import torch
        p, n = C.c_void_p(), C.c_int64()
        _check(lib().gpt_grad_arena(self.h, C.byref(p), C.byref(n)), self.h, "grad_arena")
        off = p.value - self.ws.data_ptr()
        assert off % 4 == 0 and off >= 0
        return self.ws[off:off + 4 * n.value].view(torch.float32)

    def state_arenas(self):
        """{"param", "grad", "adam_m", "adam_v": fp32, "param_bf16": bf16 or None}
        as torch views of the workspace, each of the allocated length (the
        used length is ["n"])."""
        import torch
        ptr = [C.c_void_p() for _ in range(5)]
        n, n_alloc, n_mom = C.c_int64(), C.c_int64(), C.c_int64()
        _check(lib().gpt_state_arenas(self.h, *[C.byref(x) for x in ptr], C.byref(n), C.byref(n_alloc),
                                      C.byref(n_mom)), self.h, "state_arenas")
        base = self.ws.data_ptr()

        def view(p, dtype, esize, length):
            if not p.value:
                return None
            off = p.value - base
            assert off >= 0 and off % esize == 0
            return self.ws[off:off + esize * length].view(dtype)
        out = {k: view(p, torch.float32, 4, n_alloc.value) for k, p in zip(("param", "grad"), ptr[:2])}
        out.update({k: view(p, torch.float32, 4, n_mom.value) for k, p in zip(("adam_m", "adam_v"), ptr[2:4])})
        out["param_bf16"] = view(ptr[4], torch.bfloat16, 2, n_alloc.value)
        out["n"] = int(n.value)
        out["moments_sharded"] = self.cfg.zero_world > 1
        return out

    def grad_sumsq_shard(self, offset: int, count: int, partials):
        """NORM_PARTIALS fp64 partial sums of squares of gradient elements
        [offset, offset + count) into the device tensor `partials`."""
        assert partials.numel() >= NORM_PARTIALS and partials.dtype.itemsize == 8
        _check(lib().gpt_grad_sumsq_shard(self.h, offset, count, _ptr(partials)), self.h, "grad_sumsq_shard")

    def clip_adamw_shard(self, lr: float, step: int, offset: int, count: int, grad_scale: float, partials,
                         sync: bool = True) -> Optional[float]:
        """Clip + AdamW on one shard; the global norm from the gathered partials."""
        out = C.c_float()
        _check(lib().gpt_clip_adamw_shard(self.h, lr, step, offset, count, grad_scale, _ptr(partials),
                                          partials.numel(), C.byref(out) if sync else None), self.h,
               "clip_adamw_shard")
        return float(out.value) if sync else None

    def gather_batch(self, stream_tokens, data_seed: int, step: int, micro: int, idx, tgt):
        _check(lib().gpt_gather_batch(self.h, _ptr(stream_tokens), stream_tokens.numel(), data_seed, step, micro,
                                      _ptr(idx), _ptr(tgt)), self.h, "gather_batch")

    def set_dropout_cursor(self, step: int, micro: int):
        _check(lib().gpt_set_dropout_cursor(self.h, step, micro), self.h, "set_dropout_cursor")

    def eval_loss(self, stream_tokens, data_seed: int, n_batches: int) -> float:
        """Mean loss of n_batches evaluation batches (forward only, no dropout)."""
        out = C.c_float()
        _check(lib().gpt_eval_loss(self.h, _ptr(stream_tokens), stream_tokens.numel(), data_seed, n_batches,
                                   C.byref(out)), self.h, "eval_loss")
        return float(out.value)

    def generate(self, prompt, n_new: int, temperature: float, top_k: int, top_p: float, uniform, out):
        """prompt: device int32 [batch_size, T0]; uniform: device fp32 [n_new, batch_size];
        out: device int32 [batch_size, T0 + n_new]."""
        _check(lib().gpt_generate(self.h, _ptr(prompt), prompt.shape[1], n_new, temperature, top_k, top_p,
                                  _ptr(uniform), _ptr(out)), self.h, "generate")

    def generate_kv8(self, cache: "KV8Cache", prompt, n_new: int, uniform, out, prompt_len=None, budget: int = 0,
                     recent: int = 0, table_out=None, kept=None, temperature=None, top_k=None, top_p=None, min_p=None,
                     logp=None) -> int:
        """gpt_generate_kv8.  cache: n_layer * batch_size sequences; prompt: device int32 [batch_size, T0]; prompt_len:
        int32 [batch_size]; uniform: float32 [n_new, batch_size]; out int32 and logp float32 [batch_size, n_new];
        temperature, top_p, min_p float32, top_k int32: [batch_size]; with budget > 0, table_out int32 like the cache's
        table and kept int32 [sequences, heads, budget].  Returns how often it evicted; after an odd number the cache's
        table is table_out."""
        import torch
        B = self.cfg.batch_size
        f32, i32 = torch.float32, torch.int32
        _require(prompt.dim() == 2 and cache.n_seq == self.cfg.n_layer * B,
                 "generate_kv8: prompt is [batch_size, T0], the cache has n_layer * batch_size sequences")
        for t, shape, dtype, name in ((prompt, (B, prompt.shape[1]), i32, "prompt"), (prompt_len, (B,), i32, "prompt_len"),
                                      (uniform, (n_new, B), f32, "uniform"), (out, (B, n_new), i32, "out"),
                                      (logp, (B, n_new), f32, "logp"), (temperature, (B,), f32, "temperature"),
                                      (top_k, (B,), i32, "top_k"), (top_p, (B,), f32, "top_p"), (min_p, (B,), f32, "min_p"),
                                      (table_out, tuple(cache.table.shape), i32, "table_out"),
                                      (kept, (cache.n_seq, cache.n_head_kv, budget), i32, "kept")):
            _require(t is None or (tuple(t.shape) == shape and t.dtype == dtype and t.is_contiguous() and
                                   t.device == cache.device), f"generate_kv8: {name} has another shape, type, layout or device")
        n = C.c_int32()
        _check(lib().gpt_generate_kv8(self.h, cache._ref, _ptr(prompt), _ptr(prompt_len), prompt.shape[1], n_new, budget,
                                      recent, _ptr(table_out), _ptr(kept), _ptr(temperature), _ptr(top_k), _ptr(top_p),
                                      _ptr(min_p), _ptr(uniform), _ptr(out), _ptr(logp), C.byref(n)), self.h, "generate_kv8")
        if n.value % 2:
            cache.table = table_out
        return n.value

    # -- LoRA adapters on the fused QKV blocks (targets: 1 q, 2 k, 4 v)
    def lora_attach(self, r: int, alpha: float, targets: int, A):
        """A: host float32 [blocks, r, d] (the adapted blocks' A; B starts at 0).
        Allocates the adapter workspace as a torch tensor owned by the model."""
        import torch
        n = C.c_size_t(0)
        _check(lib().gpt_lora_workspace_bytes(C.byref(self.cfg), r, targets, C.byref(n)), self.h, "lora_workspace")
        self.lora_ws = torch.empty(int(n.value), dtype=torch.uint8, device=self.device)
        A = np.ascontiguousarray(A, np.float32)
        _check(lib().gpt_lora_attach(self.h, r, alpha, targets, A.ctypes.data_as(C.c_void_p), self.lora_ws.data_ptr(),
                                     self.lora_ws.numel()), self.h, "lora_attach")
        self.lora_n = int(np.prod(A.shape)) * 2

    def lora_detach(self):
        _check(lib().gpt_lora_detach(self.h), self.h, "lora_detach")
        self.lora_ws = None

    def lora_read(self, which: int = 0) -> np.ndarray:
        out = np.empty(self.lora_n, np.float32)
        _check(lib().gpt_lora_read(self.h, which, out.ctypes.data_as(C.c_void_p), out.size), self.h, "lora_read")
        return out

    def lora_write(self, params):
        params = np.ascontiguousarray(params, np.float32)
        _check(lib().gpt_lora_write(self.h, params.ctypes.data_as(C.c_void_p), params.size), self.h, "lora_write")

    def set_graphs(self, on: bool):
        """CUDA-graph replay of train_step / train_step_host / generate (default on)."""
        _check(lib().gpt_set_graphs(self.h, 1 if on else 0), self.h, "set_graphs")

    # -- introspection
    def tensors(self) -> List[Tuple[str, Tuple[int, int]]]:
        n = C.c_int32()
        _check(lib().gpt_num_tensors(self.h, C.byref(n)), self.h)
        out = []
        for i in range(n.value):
            name = C.c_char_p()
            shape = (C.c_int64 * 2)()
            _check(lib().gpt_tensor_info(self.h, i, C.byref(name), shape), self.h)
            out.append((name.value.decode(), (int(shape[0]), int(shape[1]))))
        return out

    def get(self, kind: int = GPT_PARAM) -> Dict[str, np.ndarray]:
        res = {}
        for i, (name, (r, c)) in enumerate(self.tensors()):
            a = np.empty(r * c, dtype=np.float32)
            _check(lib().gpt_get_tensor(self.h, i, kind, a.ctypes.data), self.h, "get_tensor")
            res[name] = a.reshape((r, c) if c > 1 else (r,))
        return res

    def set(self, values: Dict[str, np.ndarray], kind: int = GPT_PARAM):
        for i, (name, (r, c)) in enumerate(self.tensors()):
            if name in values:
                a = np.ascontiguousarray(values[name], dtype=np.float32).reshape(-1)
                assert a.size == r * c, name
                _check(lib().gpt_set_tensor(self.h, i, kind, a.ctypes.data), self.h, "set_tensor")

    def logits(self) -> np.ndarray:
        a = np.empty((self.M, self.cfg.vocab_size), dtype=np.float32)
        _check(lib().gpt_get_logits(self.h, a.ctypes.data), self.h, "get_logits")
        return a

    def argmax(self) -> np.ndarray:
        a = np.empty(self.M, dtype=np.int32)
        _check(lib().gpt_get_argmax(self.h, a.ctypes.data), self.h, "get_argmax")
        return a

    def argmax_rows(self, d_rows) -> np.ndarray:
        rows, cols = d_rows.shape
        a = np.empty(rows, dtype=np.int32)
        _check(lib().gpt_argmax_rows(self.h, _ptr(d_rows), rows, cols, a.ctypes.data), self.h, "argmax_rows")
        return a

    def lse(self) -> np.ndarray:
        a = np.empty(self.M, dtype=np.float32)
        _check(lib().gpt_get_lse(self.h, a.ctypes.data), self.h, "get_lse")
        return a

    def embed_routing(self):
        n = C.c_int32()
        tok = np.empty(self.M, dtype=np.int32)
        pos = np.empty(self.M, dtype=np.int32)
        _check(lib().gpt_get_embed_routing(self.h, C.byref(n), tok.ctypes.data, pos.ctypes.data), self.h)
        return int(n.value), tok, pos

    def dropout_mask(self, counter: int, layer: int, site: int, n: int) -> np.ndarray:
        a = np.empty(n, dtype=np.uint8)
        _check(lib().gpt_dropout_mask(self.h, counter, layer, site, n, a.ctypes.data), self.h, "dropout_mask")
        return a.astype(bool)

    def get_state(self):
        n = int(lib().gpt_state_floats(self.h))
        p, m, v = (np.empty(n, dtype=np.float32) for _ in range(3))
        _check(lib().gpt_get_state(self.h, p.ctypes.data, m.ctypes.data, v.ctypes.data), self.h, "get_state")
        return p, m, v

    def set_state(self, p, m, v):
        _check(lib().gpt_set_state(self.h, _ptr(np.ascontiguousarray(p, np.float32)),
                                   _ptr(np.ascontiguousarray(m, np.float32)),
                                   _ptr(np.ascontiguousarray(v, np.float32))), self.h, "set_state")

    def flags(self) -> int:
        f = C.c_uint32()
        _check(lib().gpt_read_flags(self.h, C.byref(f)), self.h)
        return int(f.value)

    def clear_flags(self):
        _check(lib().gpt_clear_flags(self.h), self.h)

    def enable_timing(self, on: bool):
        _check(lib().gpt_enable_timing(self.h, 1 if on else 0), self.h)

    def kernel_times(self) -> Dict[str, Tuple[float, int]]:
        cap = 256
        names = (C.c_char_p * cap)()
        ms = (C.c_float * cap)()
        ln = (C.c_int32 * cap)()
        n = C.c_int32()
        _check(lib().gpt_kernel_times(self.h, cap, names, ms, ln, C.byref(n)), self.h)
        return {names[i].decode(): (float(ms[i]), int(ln[i])) for i in range(n.value)}

    def launch_count(self) -> int:
        return int(lib().gpt_launch_count(self.h))


def sample(logits, temperature: float, top_k: int, top_p: float, uniform, out, V=None, stream=None):
    """One draw per row of a device logits tensor [rows, ld] (bf16 or fp32);
    uniform: device fp32 [rows]; out: device int32 [rows]."""
    import torch
    rows, ld = logits.shape
    st = stream if stream is not None else torch.cuda.current_stream().cuda_stream
    _check(lib().gpt_sample(_ptr(logits), 1 if logits.dtype == torch.bfloat16 else 0, rows, V or ld, ld, temperature,
                            top_k, top_p, _ptr(uniform), _ptr(out), st), None, "sample")


def sample_rows(logits, uniform, out, temperature=None, top_k=None, top_p=None, min_p=None, logp=None, V=None):
    """gpt_sample_rows on the logits' device and its current stream: one draw per row of logits [rows, ld] (bf16 or
    fp32, contiguous rows).  uniform, temperature, top_p, min_p, logp: float32 [rows]; out, top_k: int32 [rows]."""
    import torch
    kind = {torch.bfloat16: 1, torch.float32: 0}.get(logits.dtype)
    if logits.dim() != 2 or kind is None or logits.stride(1) != 1:
        raise GptError(1, "sample_rows: logits are [rows, ld] of bfloat16 or float32 with contiguous rows")
    shape, dev = logits.shape, logits.get_device()
    rows, cols = shape
    V = V or cols
    ld = logits.stride(0)
    if rows == 1:
        ld = max(ld, cols)
    if V > cols or ld < cols or dev < 0:
        raise GptError(1, "sample_rows: more columns than the logits have, rows that overlap, or no device tensor")
    want, f32, i32, ptr = shape[:1], torch.float32, torch.int32, []
    for t, dtype in ((temperature, f32), (top_k, i32), (top_p, f32), (min_p, f32), (uniform, f32), (out, i32), (logp, f32)):
        if t is None:
            ptr.append(None)
        elif t.dtype is dtype and t.shape == want and t.is_contiguous() and t.get_device() == dev:
            ptr.append(t.data_ptr())
        else:
            raise GptError(1, "sample_rows: parameters are contiguous [rows] arrays (float32; top_k and out int32) on the "
                              "logits' device")
    _run_on(dev, lib().gpt_sample_rows, "sample_rows", logits.data_ptr(), kind, rows, V, ld, *ptr)


def _run_on(dev: int, fn, what: str, *args):
    """A call of the library on device dev and its current stream, which is fn's last argument."""
    import torch
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        _check(st, None, what)


def _require(cond: bool, msg: str):
    if not cond:
        raise GptError(1, msg)


class KV8Cache:
    """An 8-bit key / value cache (gpt_kv8_cache) in the caller's tensors.

    k, v: uint8 or float8_e4m3fn [n_blocks, n_head_kv, block_tokens, head_dim];
    k_scale, v_scale: float32 [n_blocks, n_head_kv]; table: int32 [n_seq,
    max_blocks]; length: int32 [n_seq]; weight (needed for accumulate and
    evict): float32 [n_blocks, n_head_kv, block_tokens]; flags: int32 [1].  All
    contiguous, on one device.  ``allocate`` makes them, with the blocks dealt
    out in order.  Calls run on the device's current stream."""

    def __init__(self, k, v, k_scale, v_scale, table, length, weight=None, flags=None):
        import torch
        e4m3 = torch.float8_e4m3fn
        _require(k.dim() == 4 and table.dim() == 2, "kv8: k is [blocks, heads, tokens, dim], table [sequences, blocks]")
        _require(k.is_cuda, "kv8: the cache is in device memory")
        for t, shape, dtypes, name in ((k, k.shape, (torch.uint8, e4m3), "k"), (v, k.shape, (torch.uint8, e4m3), "v"),
                                       (k_scale, k.shape[:2], (torch.float32,), "k_scale"),
                                       (v_scale, k.shape[:2], (torch.float32,), "v_scale"),
                                       (table, table.shape, (torch.int32,), "table"),
                                       (length, table.shape[:1], (torch.int32,), "length"),
                                       (weight, k.shape[:3], (torch.float32,), "weight"),
                                       (flags, (1,), (torch.int32,), "flags")):
            if t is not None:
                _require(tuple(t.shape) == tuple(shape) and t.dtype in dtypes and t.is_contiguous() and
                         t.device == k.device, f"kv8: {name} has another shape, type, layout or device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.length, self.weight, self.flags, self.device = length, weight, flags, k.device
        self.n_seq, self.n_head_kv, self.head_dim = table.shape[0], k.shape[1], k.shape[3]
        self._c = Kv8CacheStruct(table.shape[0], k.shape[1], k.shape[3], k.shape[2], k.shape[0], table.shape[1],
                                 _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(weight), _ptr(table),
                                 _ptr(length), _ptr(flags))
        self._ref = C.addressof(self._c)
        self._lib = lib()
        self._index, self._kind, self._i32, self._f32 = k.get_device(), {torch.bfloat16: 1, torch.float32: 0}, torch.int32, \
            torch.float32
        self._table = table

    @classmethod
    def allocate(cls, n_seq, n_head_kv, head_dim, block_tokens, max_blocks, n_blocks=None, weight=False, device="cuda"):
        """A cache with memory of its own: empty, sequence s at blocks s * max_blocks .."""
        import torch
        n = n_seq * max_blocks if n_blocks is None else n_blocks
        _require(n >= n_seq * max_blocks, "kv8: fewer blocks than the table needs")

        def zeros(*shape, dtype=torch.float32):
            return torch.zeros(*shape, dtype=dtype, device=device)
        shape = (n, n_head_kv, block_tokens, head_dim)
        table = torch.arange(n_seq * max_blocks, dtype=torch.int32, device=device).reshape(n_seq, max_blocks)
        return cls(zeros(*shape, dtype=torch.uint8), zeros(*shape, dtype=torch.uint8), zeros(n, n_head_kv),
                   zeros(n, n_head_kv), table, zeros(n_seq, dtype=torch.int32),
                   zeros(*shape[:3]) if weight else None, zeros(1, dtype=torch.int32))

    @property
    def table(self):
        return self._table

    @table.setter
    def table(self, t):
        import torch
        _require(t.dim() == 2 and t.shape[0] == self.n_seq and t.dtype == torch.int32 and t.is_contiguous() and
                 t.device == self.device, "kv8: table has another shape, type, layout or device")
        self._table = t
        self._c.d_table, self._c.max_blocks = _ptr(t), t.shape[1]

    def _rows(self, x, heads, name):
        """Pitch and type (1: bf16) of rows [n, heads, head_dim] whose heads are contiguous."""
        shape, stride, kind = x.shape, x.stride(), self._kind.get(x.dtype)
        if len(shape) != 3 or heads is not None and shape[1] != heads or shape[2] != self.head_dim or stride[2] != 1 or \
                shape[1] != 1 and stride[1] != self.head_dim or kind is None or x.get_device() != self._index:
            raise GptError(1, f"kv8: {name} is [rows, heads, head_dim] of bfloat16 or float32 with contiguous heads, on the "
                              "cache's device")
        ld, row = stride[0], shape[1] * shape[2]
        if ld < row:
            if shape[0] > 1:
                raise GptError(1, f"kv8: the rows of {name} overlap")
            ld = row
        return ld, kind

    def _start(self, start):
        if start is None:
            return None
        if start.dtype is not self._i32 or tuple(start.shape) != (self.n_seq + 1,) or not start.is_contiguous() or \
                start.get_device() != self._index:
            raise GptError(1, "kv8: start is int32 [n_seq + 1] on the cache's device")
        return start.data_ptr()

    def append(self, k, v, start=None, max_new=1):
        """gpt_kv8_append: k, v [rows, n_head_kv, head_dim], one type."""
        k_ld, b = self._rows(k, self.n_head_kv, "k")
        v_ld, bv = self._rows(v, self.n_head_kv, "v")
        n = k.shape[0]
        if b != bv or v.shape[0] != n:
            raise GptError(1, "kv8: k and v have the same rows and type")
        _run_on(self._index, self._lib.gpt_kv8_append, "kv8_append", self._ref, self._start(start), n, max_new, b,
                k.data_ptr(), k_ld, v.data_ptr(), v_ld)

    def attention(self, q, out, start=None, max_new=1, lse=None, scale=None, max_len=0):
        """gpt_kv8_attention: q, out [rows, n_head, head_dim], one type; lse (optional) float32 [rows, n_head].
        scale: 1 / sqrt(head_dim) where None."""
        q_ld, b = self._rows(q, None, "q")
        n, heads, _ = q.shape
        o_ld, bo = self._rows(out, heads, "out")
        if b != bo or out.shape[0] != n:
            raise GptError(1, "kv8: q and out have the same rows and type")
        _run_on(self._index, self._lib.gpt_kv8_attention, "kv8_attention", self._ref, self._start(start), n, max_new, heads,
                b, q.data_ptr(), q_ld, self.head_dim ** -0.5 if scale is None else scale, max_len, out.data_ptr(), o_ld,
                self._lse(lse, n, heads))

    def accumulate(self, q, lse, start=None, max_new=1, scale=None, max_len=0):
        """gpt_kv8_accumulate, with the lse that ``attention`` gave for q."""
        q_ld, b = self._rows(q, None, "q")
        n, heads, _ = q.shape
        _run_on(self._index, self._lib.gpt_kv8_accumulate, "kv8_accumulate", self._ref, self._start(start), n, max_new, heads,
                b, q.data_ptr(), q_ld, self.head_dim ** -0.5 if scale is None else scale, max_len, self._lse(lse, n, heads))

    def _lse(self, lse, n, heads):
        if lse is None:
            return None
        if lse.dtype is not self._f32 or tuple(lse.shape) != (n, heads) or not lse.is_contiguous() or \
                lse.get_device() != self._index:
            raise GptError(1, "kv8: lse is float32 [rows, n_head], contiguous, on the cache's device")
        return lse.data_ptr()

    def evict(self, table_out, budget: int, recent: int, kept):
        """gpt_kv8_evict: table_out int32 [n_seq, blocks], kept int32 [n_seq, n_head_kv, budget].  Go on with
        ``cache.table = table_out`` and ``cache.advance(max_new=0, max_len=budget)``."""
        import torch
        _require(table_out.dim() == 2 and table_out.shape[0] == self.n_seq and table_out.dtype == torch.int32 and
                 table_out.is_contiguous() and table_out.device == self.device,
                 "kv8: table_out is int32 [n_seq, blocks] on the cache's device")
        _require(kept.dtype == torch.int32 and tuple(kept.shape) == (self.n_seq, self.n_head_kv, budget) and
                 kept.is_contiguous() and kept.device == self.device, "kv8: kept is int32 [n_seq, n_head_kv, budget]")
        _run_on(self._index, self._lib.gpt_kv8_evict, "kv8_evict", self._ref, table_out.data_ptr(), table_out.shape[1],
                budget, recent, kept.data_ptr())

    def advance(self, start=None, n_rows=None, max_new=1, max_len=0):
        """gpt_kv8_advance: the lengths grow by the step's rows.  n_rows None: with start, as many as it says (give the
        arrays' own number where append was to leave out offsets past it); without, one for each sequence."""
        if n_rows is None:
            n_rows = self.n_seq if start is None else 2 ** 31 - 1
        _run_on(self._index, self._lib.gpt_kv8_advance, "kv8_advance", self._ref, self._start(start), n_rows, max_new, max_len)


def test_gemm(backend, M, N, K, A, lda, a_kmajor, B, ldb, b_kmajor, epi_kind, act=0, out=None, out2=None, ldo=0,
              aux=None, bias=None, res_in=None, res_out=None, split_k=1, partial=None, stream=None, flags=None,
              colsum=None):
    return int(lib().gpt_test_gemm(backend, M, N, K, _ptr(A), lda, a_kmajor, _ptr(B), ldb, b_kmajor, epi_kind, act,
                                   _ptr(out), _ptr(out2), ldo, _ptr(aux), _ptr(bias), _ptr(res_in), _ptr(res_out),
                                   split_k, _ptr(partial), _ptr(colsum), stream, _ptr(flags)))


def test_attention(backend, backward, dtype, B, T, H, hd, qkv, o, lse, dout=None, dqkv=None, dsum=None, p=0.0,
                   seed=0, counter=0, layer=0, stream=None, flags=None, colsum=None):
    return int(lib().gpt_test_attention(backend, backward, dtype, B, T, H, hd, _ptr(qkv), _ptr(o), _ptr(lse),
                                        _ptr(dout), _ptr(dqkv), _ptr(dsum), _ptr(colsum), p, seed, counter, layer,
                                        stream, _ptr(flags)))


def test_wait_timeout(limit_ns: int, flags, gave_up, stream=None) -> int:
    """The kernels' bounded mbarrier wait with a short limit, on a barrier
    nothing arrives at; returns the status code."""
    return int(lib().gpt_test_wait_timeout(limit_ns, stream, _ptr(flags), _ptr(gave_up)))
