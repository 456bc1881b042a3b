// wi_paged8.h -- host-side declarations shared by the sources of the attention in 8 bits.
#pragma once
#include "wi_paged.h"

// Whether a call is taken as one of single tokens: on average its requests have no more tokens than a tile of few rows takes.
bool wi_paged_few(const WiPagedGeom& g, const WiPagedAttn& a);
cudaError_t wi_launch_paged_few(const WiPagedGeom& g, const WiPagedAttn& a, const WiPagedScales& s, int sms, void* scratch,
                                int* err, cudaStream_t st);
