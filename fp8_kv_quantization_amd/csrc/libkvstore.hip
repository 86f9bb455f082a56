// The translation unit of libkvstore's stores, loads and host side.  The paged
// operators record out-of-range slots and pages in the error flag of
// kvstore.hip, a device variable of its file scope, so they are compiled with
// it; the attention kernels (attention_*.hip), which get the flag's address as
// an argument, are compiled apart, one object per source type and cache format.
#include "kvstore.hip"

#include "kvstore_rows.hip"

#include "attention_host.hip"
