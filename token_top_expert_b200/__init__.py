"""B200-native sparse-MoE block decode with calibration-free top-k channel selection.

The compute path is libmsb.so (hand-written sm_100a CUDA behind the C ABI in
include/msb.h); this package only marshals arguments to it.
"""
from ._lib import MsbError, load as load_library  # noqa: F401
from .block import (  # noqa: F401
    Dims,
    HostCall,
    PackedLayer,
    Trace,
    Workspace,
    calibrate_threshold,
    moe_sparse_block,
    moe_sparse_block_noalloc,
    moe_sparse_block_threshold,
    noalloc_check,
    pack,
    pack_q4,
    q4_record_bytes,
    path_info,
    residual_rmsnorm,
    sketch_words,
    workspace_size,
)
from .dense import (  # noqa: F401
    DenseWorkspace,
    Int8Layer,
    Routing,
    block_norm,
    combine,
    dense_check,
    grouped_matmul,
    grouped_swiglu,
    linear_int8,
    matmul_int8,
    moe_dense_block,
    quantize_int8,
    route,
    swiglu_int8,
)
from . import checkpoint, lowrank, packfile  # noqa: F401,E402
