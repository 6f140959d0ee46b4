// Internal interface between the two device translation units of libkvp.
#pragma once

// Reads and clears the device error word of kvp_sparse.cu (KVP_OK, or
// KVP_ERR_CUDA when a copy fails); kvp_check_device_error reports it.
int kvp_sparse_take_error(unsigned long long* word);
