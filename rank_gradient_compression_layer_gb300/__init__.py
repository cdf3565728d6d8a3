"""GB300-native PowerSGD compression step.

The compute lives in ``libpsgd.so`` (hand-written CUDA for sm_103a, C ABI in
``include/psgd.h``); this package only builds it and binds it with ctypes.
Beside the step: the products of expert layers (``experts_*``) and the global
gradient norm with clipping (``grad_norm``, ``clip_grad_norm``,
``GradientLayout``), the cross entropy over a vocabulary
(``linear_cross_entropy``), ``dropout`` and ``rms_norm``.
"""
from .binding import (  # noqa: F401
    EXPORTS, LIB_PATH, PHASES, PSGD_ERR_CUDA, PSGD_ERR_INVALID, PSGD_ERR_OOM, PSGD_ERR_STATE, PSGD_ERR_TIMEOUT,
    PSGD_BF16, PSGD_F16, PSGD_F32, PSGD_GRAD_NORM_WORKSPACE, PSGD_MAX_EXPERTS, PSGD_OK, PSGD_POWERSGD, PSGD_RTOPK,
    PowerSGD, PsgdError, lib, psgd_count_sent, psgd_plan_layout, psgd_plan_one_pass, psgd_plan_queue, step_noalloc,
)
from .build import build  # noqa: F401
from .language import (  # noqa: F401
    dropout, dropout_state, linear_cross_entropy, linear_cross_entropy_grad, rms_norm, rms_norm_grad,
)
from .operators import (  # noqa: F401
    GradientLayout, clip_grad_norm, experts_forward, experts_grad_input, experts_grad_weight, experts_linear,
    experts_sync, grad_norm,
)
