"""GB300 (sm_103a) kernels for the memory-bound elementwise hot path of
LTX-2-style video diffusion transformers.

* :func:`residual_gate_add` -- ``hidden + update * gate`` (full or [B, 1, D] gate)
* :func:`rmsnorm_modulate` -- ``rms_norm(x, eps) * (1 + scale) + shift``
* :func:`gate_add_rmsnorm_modulate` -- both in one pass
* :func:`rmsnorm_modulate_fp8`, :func:`gate_add_rmsnorm_modulate_fp8` -- the
  modulated output quantised to FP8 (OCP E4M3) with a per-tensor scale
* :func:`gelu_tanh` -- the feed-forward's tanh-GELU
* ``*_grouped`` -- the first three over several problems (e.g. the video and
  audio streams of a block) in one launch
* :func:`selfcheck` / :func:`ensure_checked` -- bit-for-bit check of one
  runtime key (op, dtype, layouts, D) on the GPU
* :func:`set_statistic` / :func:`statistic` -- the modulation's row
  statistic: "fast" (default) or "exact" (correctly rounded, bit-exact)
* :func:`rmsnorm`, :func:`add_rmsnorm`, :func:`rmsnorm_fp8`,
  :func:`add_rmsnorm_fp8` -- the weighted RMSNorm of token transformers, with
  the residual's addition and an E4M3 output with dynamic scales
* :func:`rmsnorm_backward` -- its gradients
* :func:`embedding`, :func:`embedding_backward` -- rows of a table by token
  id, and the table's gradient by sorted tokens
* :func:`grad_norm`, :func:`clip_grads`, :class:`TensorList` -- the 2-norm over
  many tensors, and clipping by it
* :func:`rotary_frequencies`, :func:`rotary_table` -- cos and sin of the
  angles of positions, over one or several axes
* :func:`rope`, :func:`rmsnorm_rope`, :func:`rmsnorm_rope_backward` -- queries
  and keys turned by them, with the norm of each head in the same pass, and
  the gradients
* :class:`KVCache`, :func:`cache_write`, :func:`cache_read`,
  :func:`paged_attention` -- a paged cache of keys and values (E4M3 with a
  scale per row, or in the dtype), and the attention of one new token per
  sequence over it

Each call is one kernel of ``libdit_elementwise.so`` (C ABI in
``include/dit_elementwise.h``), launched on the current torch stream; the
gradients, the norm over tensors and the paged attention are a few.  Build
the library with :func:`build`; without it every call raises.
"""
from ._attend import (  # noqa: F401
    KVCache,
    cache_read,
    cache_write,
    paged_attention,
    rmsnorm_rope,
    rmsnorm_rope_backward,
    rope,
    rotary_frequencies,
    rotary_table,
)
from ._binding import (  # noqa: F401
    DitError,
    ensure_checked,
    gate_add_rmsnorm_modulate,
    gate_add_rmsnorm_modulate_fp8,
    gate_add_rmsnorm_modulate_grouped,
    gelu_tanh,
    library,
    residual_gate_add,
    residual_gate_add_grouped,
    rmsnorm_modulate,
    rmsnorm_modulate_fp8,
    rmsnorm_modulate_grouped,
    get_statistic,
    selfcheck,
    set_first_use_check,
    set_statistic,
    statistic,
)
from ._token import (  # noqa: F401
    TensorList,
    add_rmsnorm,
    add_rmsnorm_fp8,
    clip_grads,
    embedding,
    embedding_backward,
    grad_norm,
    rmsnorm,
    rmsnorm_backward,
    rmsnorm_fp8,
)
from .build import build  # noqa: F401
