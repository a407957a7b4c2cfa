// qsa_lib.cu -- the one translation unit of libqsa.so.
#include "qsa_api.cu"
#include "qsa_state.cuh"
