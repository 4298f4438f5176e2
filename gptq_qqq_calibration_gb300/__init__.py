"""GB300-native accumulation of the GPTQ/QQQ calibration Hessian.

``H = (2/N) sum_t x_t x_t^T`` over ragged batches of layer-input activations
(N counts tokens), damped by ``damp_percent * mean(diag H)`` when it is
materialized, plus the batched 16x16 per-block "local Hessian", and the
quantization pass that consumes H (``GPTQ``).  Next to them: the gated
feed-forward projections that make the down projection's input, and their
gradient (``GatedFF``), the distillation loss of a quantized model from its
original's top logits (``distill_*``), 8-bit rows (``quantize_rows``), which keep
activations for a backward pass, and the 8-bit integer linear layer with its
gradient (``Int8Linear``), which runs a quantized layer.  All of the arithmetic runs in the CUDA
library ``libgptq_hess.so`` (sm_103a) behind the C ABI in ``include/``; this
package only marshals arguments.
"""

from .hessian import *  # noqa: F401,F403
from .hessian import Hessian, IMatrix, LocalHessian  # noqa: F401
from .gptq import GPTQ  # noqa: F401
from .distill import distill_backward, distill_forward, distill_loss, distill_step  # noqa: F401
from .gated_ff import GatedFF  # noqa: F401
from .int8_linear import Int8Linear  # noqa: F401
from .rows8 import Rows8, quantize_rows, restore_rows  # noqa: F401
